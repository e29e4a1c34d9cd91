// gfx950 kernels of the layers' products for at most 16 rows (tokens that are being
// decoded): C[m][n] = sum_k A[m][k] B[n][k] is then bound by reading B once.
//
// A workgroup takes 16 rows of B (of both projections, in the gated block) and its
// waves blocks of K in turn, so that it reads runs of consecutive bytes of 16 rows.
// Every lane loads the 16 bytes that its MFMA operand is, straight into registers: B's
// rows are the MFMA's rows, A's its columns (past the last one the last one again).
// A wave asks for its next block before it multiplies the one at hand: 8 to 16 KB in
// flight a wave. The waves' sums meet in LDS, in a fixed order. No tile is filled, no
// pieces are joined by a second launch, and any alignment will do.
//
// The other way, 64 x 64 tiles: 16.2 and 13.6 us where these take @ and @ (one token, 2048 x
// 6144 weights), @.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mlp_math.h"
#include "product.h"

namespace muon {

constexpr int kFewWaves = 16;  // at most

// A block of K of one wave: so many steps of an MFMA's K that two blocks fit its 128
// registers.
template <int BYTES>  // of an element
constexpr int kFewSteps = BYTES == 2 ? 4 : 2;

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
    float t[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) cut3(v[i], t[2][i], t[1][i], t[0][i]);
#pragma unroll
    for (int q = 0; q < 3; ++q)
      o[q] = __builtin_bit_cast(bf16x8, (u32x4{pack_bf16x2(t[q][0], t[q][1]), pack_bf16x2(t[q][2], t[q][3]),
                                               pack_bf16x2(t[q][4], t[q][5]), pack_bf16x2(t[q][6], t[q][7])}));
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
// the workgroup's). An MFMA's element r of lane l is B's row 4 (l / 16) + r, A's l % 16.
template <int OPS>
MUON_INLINE void few_join(float (&red)[kFewWaves][OPS][256], const f32x4 (&acc)[OPS], float v[OPS]) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
#pragma unroll
  for (int o = 0; o < OPS; ++o)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][o][(lane & 15) * 16 + 4 * (lane >> 4) + r] = acc[o][r];
  __syncthreads();
#pragma unroll
  for (int o = 0; o < OPS; ++o) v[o] = 0.f;
  if (tid < 256)
    for (int w = 0; w < waves; ++w)
#pragma unroll
      for (int o = 0; o < OPS; ++o) v[o] += red[w][o][tid];
}

// bf16 or fp32. OPS 2: s = act(a) * b; 1: the product itself.
template <class T, int OPS>
__global__ void __launch_bounds__(64 * kFewWaves) few_kernel(FewArgs p) {
  typedef FewRun<T> Run;
  __shared__ float red[kFewWaves][OPS][256];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
  const int n0 = blockIdx.x * 16, q = lane >> 4;
  const T* xr = static_cast<const T*>(p.a) + (int64_t)min(lane & 15, p.m - 1) * p.lda;
  const T* wr[OPS];
#pragma unroll
  for (int o = 0; o < OPS; ++o) wr[o] = static_cast<const T*>(p.b[o]) + (int64_t)min(n0 + (lane & 15), p.n - 1) * p.ldb;
  f32x4 acc[OPS];
#pragma unroll
  for (int o = 0; o < OPS; ++o) acc[o] = f32x4{0.f, 0.f, 0.f, 0.f};
  constexpr int STEPS = kFewSteps<sizeof(T)>, KB = 32 * STEPS;
  const int blocks = p.k / KB;
  struct Block {
    Run x[STEPS], w[OPS][STEPS];
  };
  auto load = [&](Block& b, int i) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int64_t k = (int64_t)i * KB + 32 * s + 8 * q;
#pragma unroll
      for (int o = 0; o < OPS; ++o) b.w[o][s].load(wr[o] + k);
      b.x[s].load(xr + k);
    }
  };
  auto sum = [&](const Block& b) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      bf16x8 x[Run::PARTS], w[Run::PARTS];
      b.x[s].operands(x);
#pragma unroll
      for (int o = 0; o < OPS; ++o) {
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
      Run x, w[OPS];
      x.load_tail(xr + min(k, p.k - 1), p.k - k);
      bf16x8 xo[Run::PARTS], wo[Run::PARTS];
      x.operands(xo);
#pragma unroll
      for (int o = 0; o < OPS; ++o) {
        w[o].load_tail(wr[o] + min(k, p.k - 1), p.k - k);
        w[o].operands(wo);
        acc[o] = few_mfma<Run::PARTS>(wo, xo, acc[o]);
      }
    }
  }
  float v[OPS];
  few_join<OPS>(red, acc, v);
  const int row = tid >> 4, col = n0 + (tid & 15);
  if (tid >= 256 || row >= p.m || col >= p.n) return;
  float y = v[0];
  if constexpr (OPS == 2) y = activation(v[0], p.act) * v[1];
  T* out = static_cast<T*>(p.out) + (int64_t)row * p.ldo + col;
  if (p.beta != 0.f) y += p.beta * Elem<T>::load(static_cast<const T*>(p.c) + (int64_t)row * p.ldc + col);
  Elem<T>::store(out, y);
}

// e4m3 operands with scales, results in bf16. A step is the 8-bit MFMA's 128 of K; a lane's operand is bytes 16 q .. and 64 + 16 q .. of a step, its scale that
// of bytes 32 q ...
__global__ void __launch_bounds__(64 * kFewWaves) few8_kernel(FewArgs p) {
  __shared__ float red[kFewWaves][1][256];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
  const int n0 = blockIdx.x * 16, q = lane >> 4;
  const int row = min(lane & 15, p.m - 1);
  const uint8_t* xr = static_cast<const uint8_t*>(p.a) + (int64_t)row * p.lda;
  const uint8_t* xe = p.ea + (int64_t)row * p.lde;
  const uint8_t* wr = static_cast<const uint8_t*>(p.b[0]) + (int64_t)min(n0 + (lane & 15), p.n - 1) * p.ldb;
  const uint8_t* we = p.eb + n0 / kBlock * p.ldeb_n;
  f32x4 acc[1] = {f32x4{0.f, 0.f, 0.f, 0.f}};
  constexpr int STEPS = kFewSteps<1>, KB = kBlock * STEPS;
  const int blocks = p.k / KB, groups = (p.k + kGroup - 1) / kGroup;
  struct Block {
    u32x4 x[STEPS][2], w[STEPS][2];
    uint32_t ex[STEPS], ew[STEPS];
  };
  auto load = [&](Block& b, int i) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int64_t k = (int64_t)i * KB + kBlock * s;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        b.w[s][h] = gload16(wr + k + 64 * h + 16 * q);
        b.x[s][h] = gload16(xr + k + 64 * h + 16 * q);
      }
      b.ex[s] = *((const g_u8*)(xe + k / kGroup + q));
      b.ew[s] = *((const g_u8*)(we + k / kBlock * p.ldeb_k));
    }
  };
  auto join = [&](const u32x4 v[2]) __attribute__((always_inline)) {
    return i32x8{(int)v[0][0], (int)v[0][1], (int)v[0][2], (int)v[0][3], (int)v[1][0], (int)v[1][1], (int)v[1][2], (int)v[1][3]};
  };
  auto sum = [&](const Block& b) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
      acc[0] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(b.w[s]), join(b.x[s]), acc[0], 0, 0, 0, (int)b.ew[s], 0, (int)b.ex[s]);
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
    auto half = [&](const uint8_t* r, int k) __attribute__((always_inline)) {
      u32x4 v = gload16(r + min(k, padded - 16));
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int b = p.k - k - 4 * w;
        v[w] &= b >= 4 ? ~0u : b <= 0 ? 0u : (1u << (8 * b)) - 1u;
      }
      return v;
    };
#pragma unroll 1
    for (int k = blocks * KB; k < p.k; k += kBlock) {
      const u32x4 w[2] = {half(wr, k + 16 * q), half(wr, k + 64 + 16 * q)}, x[2] = {half(xr, k + 16 * q), half(xr, k + 64 + 16 * q)};
      const int g = k / kGroup + q;
      const uint32_t ex = g < groups ? (uint32_t)*((const g_u8*)(xe + g)) : 127u;
      const uint32_t ew = *((const g_u8*)(we + k / kBlock * p.ldeb_k));
      acc[0] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(w), join(x), acc[0], 0, 0, 0, (int)ew, 0, (int)ex);
    }
  }
  float v[1];
  few_join<1>(red, acc, v);
  const int m = tid >> 4, col = n0 + (tid & 15);
  if (tid >= 256 || m >= p.m || col >= p.n) return;
  if (p.beta != 0.f) v[0] += p.beta * Elem<u16>::load(static_cast<const u16*>(p.c) + (int64_t)m * p.ldc + col);
  Elem<u16>::store(static_cast<u16*>(p.out) + (int64_t)m * p.ldo + col, v[0]);
}

// Workgroups of 16 waves where there are fewer than CUs, else of 8 (two projections of
// 6144 x 2048: 12.1 us, with 16 waves 13.9; one of 2048 x 6144 8.6 with 16).
static dim3 few_block(const FewArgs& a) { return dim3(64 * ((a.n + 15) / 16 < 256 ? kFewWaves : kFewWaves / 2)); }

hipError_t launch_few(const FewArgs& a, bool f32, int ops, hipStream_t s) {
  const dim3 grid((uint32_t)((a.n + 15) / 16)), block = few_block(a);
  if (ops == 2) {
    if (f32) hipLaunchKernelGGL((few_kernel<float, 2>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((few_kernel<u16, 2>), grid, block, 0, s, a);
  } else {
    if (f32) hipLaunchKernelGGL((few_kernel<float, 1>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((few_kernel<u16, 1>), grid, block, 0, s, a);
  }
  return hipGetLastError();
}

hipError_t launch_few8(const FewArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(few8_kernel, dim3((uint32_t)((a.n + 15) / 16)), few_block(a), 0, s, a);
  return hipGetLastError();
}

}  // namespace muon
