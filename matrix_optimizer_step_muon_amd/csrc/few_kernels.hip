// gfx950 kernels of the layers' products for at most 16 rows (tokens that are being
// decoded): C[m][n] = sum_k A[m][k] B[n][k] is then bound by reading B once.
//
// A workgroup takes up to 32 rows of B (of both projections, in the gated block) and
// its waves blocks of K in turn, so that it reads runs of consecutive bytes of these
// rows. So many rows that every CU gets the same share: 16 always would leave 64 of
// 256 CUs with twice the others' work at 5120 rows, and half of them without at 2048
// (8-bit weights of 5120 x 25600 then take 32.9 us, and 24.4 as it is; in bf16 2048 x
// 6144 9.0 and 7.1, both projections of 25600 x 5120 97.4 and 89.0: the first two from the
// last-level cache, from HBM 28.5, 4.6 TB/s, and 8.4; the last, 5.9 TB/s, from HBM). Every
// lane loads the 16 bytes that its MFMA operand is, straight into registers: B's rows
// are the MFMA's rows, A's its columns (past the last one the last one again). A wave
// asks for its next block before it multiplies the one at hand: 8 to 16 KB in flight a
// wave. The waves' sums meet in LDS, in a fixed order. No tile is filled, no pieces
// are joined by a second launch, and any alignment will do.
//
// The other way, 64 x 64 tiles: 16.2 and 13.6 us where these take 10.8 and 7.1 (one
// token, both projections of 6144 x 2048 and the down projection).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mlp_math.h"
#include "product.h"

namespace muon {

constexpr int kFewWaves = 16;  // at most

// A block of K of one wave: so many steps of an MFMA's K that two blocks fit its 128
// registers. WAYS: operands of B's kind.
template <int BYTES, int WAYS>  // of an element
constexpr int kFewSteps = BYTES == 2 ? (WAYS <= 2 ? 4 : 2) : BYTES == 4 ? 2 : WAYS == 1 ? 2 : 1;

// 8 consecutive elements of a row as an MFMA operand: one, or in fp32 the three bf16
// operands that add up to it.
template <class T>
struct FewRun;
template <>
struct FewRun<u16> {
  static constexpr int PARTS = 1;
  u32x4 v;
  MUON_INLINE void load(const u16* p) { v = gload16_any(p); }
  MUON_INLINE void load_tail(const u16* p, int live) {  // of 8, the first `live`; 0 past them
    u16 t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = i < live ? (u16)*((const g_u16*)(p + i)) : (u16)0;
    v = __builtin_bit_cast(u32x4, t);
  }
  MUON_INLINE void operands(bf16x8 o[1]) const { o[0] = __builtin_bit_cast(bf16x8, v); }
};
template <>
struct FewRun<float> {
  static constexpr int PARTS = 3;
  float v[8];
  MUON_INLINE void load(const float* p) {
    const u32x4 lo = gload16_any(p), hi = gload16_any(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(lo[i]);
      v[4 + i] = __uint_as_float(hi[i]);
    }
  }
  MUON_INLINE void load_tail(const float* p, int live) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < live ? Elem<float>::load(p + i) : 0.f;
  }
  MUON_INLINE void operands(bf16x8 o[3]) const {  // lo, mid, hi
    u32x4 t[3];
    cut3(v, t);
#pragma unroll
    for (int q = 0; q < 3; ++q) o[q] = __builtin_bit_cast(bf16x8, t[q]);
  }
};

// acc += a b of one step; fp32: the six products down to 2^-24 of the largest, the
// smallest first.
template <int PARTS>
MUON_INLINE f32x4 few_mfma(const bf16x8 (&b)[PARTS], const bf16x8 (&a)[PARTS], f32x4 acc) {
  if constexpr (PARTS == 1) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[0], a[0], acc, 0, 0, 0);
  } else {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[0], a[2], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[2], a[0], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[1], a[1], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[1], a[2], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[2], a[1], acc, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[2], a[2], acc, 0, 0, 0);
  }
}

// The sums of all waves, of this thread's output (row t / 16 of A, row t % 16 of B of
// each 16 of the workgroup's). An MFMA's element r of lane l is B's row 4 (l / 16) + r,
// A's l % 16. `halves`: A's rows 8 to 15 are what rows 0 to 7 have beside.
template <int WAYS>
MUON_INLINE void few_join(float (&red)[kFewWaves][WAYS][256], const f32x4 (&acc)[WAYS], float v[WAYS], bool halves = false) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
#pragma unroll
  for (int o = 0; o < WAYS; ++o)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][o][(lane & 15) * 16 + 4 * (lane >> 4) + r] = acc[o][r];
  __syncthreads();
#pragma unroll
  for (int o = 0; o < WAYS; ++o) v[o] = 0.f;
  if (halves && tid < 128)
    for (int w = 0; w < waves; ++w)
#pragma unroll
      for (int o = 0; o < WAYS; ++o) v[o] += red[w][o][tid + 128];
  if (tid < 256)
    for (int w = 0; w < waves; ++w)
#pragma unroll
      for (int o = 0; o < WAYS; ++o) v[o] += red[w][o][tid];
}

// bf16 or fp32. OPS 2: s = act(a) * b; 1: the product itself. G: sixteens of rows of B.
// Rounding s to bf16 costs as much accuracy as rounding y does. With up to kFewHalves rows
// s has a second plane with the next 8 bits in columns of the MFMA that are idle. What
// that takes is reading twice the rows of s: 2048 x 6144, weights from HBM, with one plane
// and two, 1 row 20.8 and 21.0 us, 2 rows 20.8 and 21.2, 4 rows 21.1 and 22.2, 8 rows 22.1
// and 24.3; 5120 x 25600, 1 row 137.0 and 137.6, 8 rows 147 and 159.
template <class T, int OPS, int G>
__global__ void __launch_bounds__(64 * kFewWaves) few_kernel(FewArgs p) {
  typedef FewRun<T> Run;
  constexpr int WAYS = OPS * G;  // operand OPS * g + o: the g-th sixteen of weight o
  __shared__ float red[kFewWaves][WAYS][256];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
  const int n0 = blockIdx.x * p.per, n1 = min(n0 + p.per, p.n), q = lane >> 4;
  const bool halves = OPS == 1 && sizeof(T) == 2 && p.plane;
  const T* xr = static_cast<const T*>(p.a) + (int64_t)min(halves ? lane & 7 : lane & 15, p.m - 1) * p.lda;
  if (halves && lane & 8) xr += p.plane;
  const T* wr[WAYS];
#pragma unroll
  for (int o = 0; o < WAYS; ++o)
    wr[o] = static_cast<const T*>(p.b[o % OPS]) + (int64_t)min(n0 + o / OPS * 16 + (lane & 15), n1 - 1) * p.ldb;
  f32x4 acc[WAYS];
#pragma unroll
  for (int o = 0; o < WAYS; ++o) acc[o] = f32x4{0.f, 0.f, 0.f, 0.f};
  constexpr int STEPS = kFewSteps<sizeof(T), WAYS>, KB = 32 * STEPS;
  const int blocks = p.k / KB;
  struct Block {
    Run x[STEPS], w[WAYS][STEPS];
  };
  auto load = [&](Block& b, int i) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int64_t k = (int64_t)i * KB + 32 * s + 8 * q;
#pragma unroll
      for (int o = 0; o < WAYS; ++o) b.w[o][s].load(wr[o] + k);
      b.x[s].load(xr + k);
    }
  };
  auto sum = [&](const Block& b) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      bf16x8 x[Run::PARTS], w[Run::PARTS];
      b.x[s].operands(x);
#pragma unroll
      for (int o = 0; o < WAYS; ++o) {
        b.w[o][s].operands(w);
        acc[o] = few_mfma<Run::PARTS>(w, x, acc[o]);
      }
    }
  };
  int i = wave;
  Block b0, b1;
  if (i < blocks) load(b0, i);
#pragma unroll 1
  for (; i < blocks; i += 2 * waves) {
    if (i + waves < blocks) load(b1, i + waves);
    sum(b0);
    if (i + 2 * waves < blocks) load(b0, i + 2 * waves);
    if (i + waves < blocks) sum(b1);
  }
  if (blocks * KB < p.k && wave == blocks % waves) {  // what is left of K
#pragma unroll 1
    for (int k = blocks * KB + 8 * q; k < (p.k + 31) / 32 * 32; k += 32) {
      Run x, w[WAYS];
      x.load_tail(xr + min(k, p.k - 1), p.k - k);
      bf16x8 xo[Run::PARTS], wo[Run::PARTS];
      x.operands(xo);
#pragma unroll
      for (int o = 0; o < WAYS; ++o) {
        w[o].load_tail(wr[o] + min(k, p.k - 1), p.k - k);
        w[o].operands(wo);
        acc[o] = few_mfma<Run::PARTS>(wo, xo, acc[o]);
      }
    }
  }
  float v[WAYS];
  few_join<WAYS>(red, acc, v, halves);
  const int row = tid >> 4;
  if (tid >= 256 || row >= p.m) return;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int col = n0 + 16 * g + (tid & 15);
    if (col >= n1) return;
    float y = v[OPS * g];
    if constexpr (OPS == 2) y = activation(y, p.act) * v[OPS * g + 1];
    T* to = static_cast<T*>(p.out) + (int64_t)row * p.ldo + col;
    if constexpr (OPS == 2 && sizeof(T) == 2) {
      if (p.plane) {
        u16 hi, lo;
        cut2(y, hi, lo);
        *((g_u16*)to) = hi;
        *((g_u16*)(to + p.plane)) = lo;
        continue;
      }
    }
    Elem<T>::store(to, y);
  }
}

// e4m3 operands with scales, results in bf16. A step is the 8-bit MFMA's 128 of K; a
// lane's operand is bytes 16 q .. and 64 + 16 q .. of a step, its scale that of bytes
// 32 q ...
template <int G>
__global__ void __launch_bounds__(64 * kFewWaves) few8_kernel(FewArgs p) {
  __shared__ float red[kFewWaves][G][256];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
  const int n0 = blockIdx.x * p.per, n1 = min(n0 + p.per, p.n), q = lane >> 4;
  const int row = min(lane & 15, p.m - 1);
  const uint8_t* xr = static_cast<const uint8_t*>(p.a) + (int64_t)row * p.lda + 16 * q;
  const uint8_t* xe = p.ea + (int64_t)row * p.lde;
  const uint8_t *wr[G], *we[G];
  f32x4 acc[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int n = min(n0 + 16 * g + (lane & 15), n1 - 1);
    wr[g] = static_cast<const uint8_t*>(p.b[0]) + (int64_t)n * p.ldb + 16 * q;
    we[g] = p.eb + n / kBlock * p.ldeb_n;
    acc[g] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  constexpr int STEPS = kFewSteps<1, G>, KB = kBlock * STEPS;
  const int blocks = p.k / KB, groups = (p.k + kGroup - 1) / kGroup;
  struct Block {
    u32x4 x[STEPS][2], w[G][STEPS][2];
    uint32_t ex[STEPS], ew[G][STEPS];
  };
  auto load = [&](Block& b, int i) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int64_t k = (int64_t)i * KB + kBlock * s;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int g = 0; g < G; ++g) b.w[g][s][h] = gload16(wr[g] + k + 64 * h);
        b.x[s][h] = gload16(xr + k + 64 * h);
      }
      b.ex[s] = *((const g_u8*)(xe + k / kGroup + q));
#pragma unroll
      for (int g = 0; g < G; ++g) b.ew[g][s] = *((const g_u8*)(we[g] + k / kBlock * p.ldeb_k));
    }
  };
  auto join = [&](const u32x4 v[2]) __attribute__((always_inline)) {
    return i32x8{(int)v[0][0], (int)v[0][1], (int)v[0][2], (int)v[0][3], (int)v[1][0], (int)v[1][1], (int)v[1][2], (int)v[1][3]};
  };
  auto sum = [&](const Block& b) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int g = 0; g < G; ++g)
        acc[g] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(b.w[g][s]), join(b.x[s]), acc[g], 0, 0, 0, (int)b.ew[g][s],
                                                                  0, (int)b.ex[s]);
  };
  int i = wave;
  Block b0, b1;
  if (i < blocks) load(b0, i);
#pragma unroll 1
  for (; i < blocks; i += 2 * waves) {
    if (i + waves < blocks) load(b1, i + waves);
    sum(b0);
    if (i + 2 * waves < blocks) load(b0, i + 2 * waves);
    if (i + waves < blocks) sum(b1);
  }
  if (blocks * KB < p.k && wave == blocks % waves) {
    // What is left of K, 128 at a time: rows are readable up to a multiple of 16, and
    // what is behind K becomes 0 in both operands, with a scale of 1.
    const int padded = (p.k + 15) / 16 * 16;
    auto half = [&](const uint8_t* r, int k) __attribute__((always_inline)) {  // r is 16 q on
      u32x4 v = gload16(r + (min(k, padded - 16) - 16 * q));
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int b = p.k - k - 4 * w;
        v[w] &= b >= 4 ? ~0u : b <= 0 ? 0u : (1u << (8 * b)) - 1u;
      }
      return v;
    };
#pragma unroll 1
    for (int k = blocks * KB; k < p.k; k += kBlock) {
      const u32x4 x[2] = {half(xr, k + 16 * q), half(xr, k + 64 + 16 * q)};
      const int at = k / kGroup + q;
      const uint32_t ex = at < groups ? (uint32_t)*((const g_u8*)(xe + at)) : 127u;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const u32x4 w[2] = {half(wr[g], k + 16 * q), half(wr[g], k + 64 + 16 * q)};
        const uint32_t ew = *((const g_u8*)(we[g] + k / kBlock * p.ldeb_k));
        acc[g] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(w), join(x), acc[g], 0, 0, 0, (int)ew, 0, (int)ex);
      }
    }
  }
  float v[G];
  few_join<G>(red, acc, v);
  const int m = tid >> 4;
  if (tid >= 256 || m >= p.m) return;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int col = n0 + 16 * g + (tid & 15);
    if (col >= n1) return;
    if (p.beta != 0.f) v[g] += p.beta * Elem<u16>::load(static_cast<const u16*>(p.c) + (int64_t)m * p.ldc + col);
    Elem<u16>::store(static_cast<u16*>(p.out) + (int64_t)m * p.ldo + col, v[g]);
  }
}

// Waves: 16 where every CU gets one workgroup, else 8.
struct FewGrid {
  dim3 grid, block;
};
static FewGrid few_grid(FewArgs& a, int most) {
  const FewShare f = few_share(a.n, most);
  a.per = (int)f.per;
  return {dim3((uint32_t)((a.n + f.per - 1) / f.per)), dim3(64 * (f.rounds == 1 ? kFewWaves : kFewWaves / 2))};
}

template <class T, int OPS>
static hipError_t launch_few_of(FewArgs a, hipStream_t s) {
  const FewGrid g = few_grid(a, sizeof(T) == 2 ? kFewMost : kFewMostF32);
  if (a.per <= 16) hipLaunchKernelGGL((few_kernel<T, OPS, 1>), g.grid, g.block, 0, s, a);
  else if constexpr (sizeof(T) == 2) hipLaunchKernelGGL((few_kernel<T, OPS, 2>), g.grid, g.block, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_few(const FewArgs& a, bool f32, int ops, hipStream_t s) {
  if (ops == 2) return f32 ? launch_few_of<float, 2>(a, s) : launch_few_of<u16, 2>(a, s);
  return f32 ? launch_few_of<float, 1>(a, s) : launch_few_of<u16, 1>(a, s);
}

hipError_t launch_few8(const FewArgs& args, hipStream_t s) {
  FewArgs a = args;
  const FewGrid g = few_grid(a, kFewMost);
  if (a.per <= 16) hipLaunchKernelGGL(few8_kernel<1>, g.grid, g.block, 0, s, a);
  else hipLaunchKernelGGL(few8_kernel<2>, g.grid, g.block, 0, s, a);
  return hipGetLastError();
}

}  // namespace muon
