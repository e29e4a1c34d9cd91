// gfx950 kernels of the weight gradient from an 8-bit checkpoint,
//   G[n][k] = scale[k] * sum_t dY[t][n] X[t][k]  + beta * C[n][k].
//
// The sum runs over tokens, the slow index of both operands, so both are read
// from LDS with the transposing load: token rows go into LDS as they lie in
// memory, and an MFMA operand (8 consecutive tokens of one column per lane) is
// two transposing reads. dY rows are copied straight into LDS; checkpoint bytes
// go through registers, where they become bf16. A checkpoint's scale is a power
// of two, so its values are exactly bf16 and the decoded operand loses nothing.
// fp32 dY comes as three bf16 planes (hi, mid, lo parts) summed one after the
// other, over the same checkpoint.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device.h"
#include "layer_internal.h"
#include "q8.h"

namespace muon {

// Stage geometry: 64 tokens of 256 bf16 columns per operand, two stages.
constexpr int kRowBytes = kWgTile * 2;
constexpr int kOpBytes = kWgStep * kRowBytes;  // 32 KB
constexpr int kStageBytes = 2 * kOpBytes;
constexpr int kDmaPerWave = kOpBytes / 1024 / 4;       // 8
constexpr int kChunks = kWgStep * kWgTile / 16 / 256;  // 16-byte checkpoint chunks per thread: 4

typedef const __attribute__((address_space(4))) WgArgs* ArgsPtr;

// The unit of workgroup b: XCD b % 8 gets a contiguous range of units, so that
// the tiles that run there together share operand panels in its L2.
MUON_INLINE int xcd_unit(int b, int units) {
  const int x = b & 7, i = b >> 3, per = units >> 3, rest = units & 7;
  return x * per + min(x, rest) + i;
}

// Tile (tn, tk) of local tile number t: bands of 4 tile rows walked column by
// column, so 32 consecutive tiles cover 4 x 8.
MUON_INLINE void tile_of(int t, int tiles_n, int tiles_k, int& tn, int& tk) {
  const int band = t / (4 * tiles_k), r = t - band * 4 * tiles_k;
  const int h = min(4, tiles_n - 4 * band);
  tk = r / h;
  tn = 4 * band + (r - tk * h);
}

// Four consecutive columns k .. k+3 of row n of the gradient.
MUON_INLINE void store_grad(const __attribute__((address_space(4))) WgItem& it, bool scale_f32, bool g_f32, int n, int k,
                            const float* v) {
  if (n >= it.n || k >= it.k) return;
  const int64_t at = (int64_t)n * it.k + k;
  const int cnt = min(4, it.k - k);
  float o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = v[i];
  if (it.scale) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < cnt)
        o[i] *= scale_f32 ? Elem<float>::load(static_cast<const float*>(it.scale) + k + i)
                          : Elem<u16>::load(static_cast<const u16*>(it.scale) + k + i);
  }
  const bool vec = (it.k & 3) == 0;  // g and c are 16-byte aligned, k is a multiple of 4
  if (it.beta != 0.f) {
    float c[4] = {0.f, 0.f, 0.f, 0.f};
    if (g_f32) {
      const float* p = static_cast<const float*>(it.c) + at;
      if (vec) Vec4<float>::load(p, c);
      else
        for (int i = 0; i < cnt; ++i) c[i] = Elem<float>::load(p + i);
    } else {
      const u16* p = static_cast<const u16*>(it.c) + at;
      if (vec) Vec4<u16>::load(p, c);
      else
        for (int i = 0; i < cnt; ++i) c[i] = Elem<u16>::load(p + i);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] += it.beta * c[i];
  }
  if (g_f32) {
    float* p = static_cast<float*>(it.g) + at;
    if (vec) Vec4<float>::store(p, o);
    else
      for (int i = 0; i < cnt; ++i) Elem<float>::store(p + i, o[i]);
  } else {
    u16* p = static_cast<u16*>(it.g) + at;
    if (vec) Vec4<u16>::store(p, o);
    else
      for (int i = 0; i < cnt; ++i) Elem<u16>::store(p + i, o[i]);
  }
}

template <int KIND>
__global__ void __launch_bounds__(256, 1) wgrad_kernel(WgArgs) {
  __shared__ __align__(1024) unsigned char smem[2 * kStageBytes];
  const ArgsPtr a = (ArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
  const int unit = xcd_unit(blockIdx.x, a->units);
  int idx = 0;
  while (idx + 1 < a->n_items && unit >= a->item[idx + 1].unit0) ++idx;
  const __attribute__((address_space(4))) WgItem& it = a->item[idx];
  const int tiles = it.tiles_n * it.tiles_k;
  const int local = unit - it.unit0, split = local / tiles, tile = local - split * tiles;
  int tn, tk;
  tile_of(tile, it.tiles_n, it.tiles_k, tn, tk);
  const int n0 = tn * kWgTile, k0 = tk * kWgTile;
  const int per_plane = (it.rows + kWgStep - 1) / kWgStep;
  const int total = per_plane * it.parts;
  // split s takes stages [total*s/splits, total*(s+1)/splits)
  const int s_begin = (int)((int64_t)total * split / it.splits);
  const int s_end = (int)((int64_t)total * (split + 1) / it.splits);

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  f32x16 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
  // Held in scalar registers: reloaded in the loop, they would make it wait for
  // every LDS access in flight (scalar loads share that counter).
  int rows = it.rows;
  int64_t lda = it.lda, ldq = it.ldq, lde = it.lde;
  const uint8_t *xq = it.q, *xe = it.e;
  asm volatile("" : "+s"(rows), "+s"(lda), "+s"(ldq), "+s"(lde), "+s"(xq), "+s"(xe));

  // A stage covers tokens t0 .. t0+63 of a plane. The last stage of a plane
  // may be shorter: it still reads 64 token rows, the last 64 (or, in a
  // product of fewer, the last row again), so no address depends on how many
  // are left; rows that are not the stage's own become zeros in both operands
  // (in both, because the other one may hold an infinity).
  const int last_base = max(rows - kWgStep, 0);
  struct Stage {
    const u16* dy;  // its plane's first row
    int t0;
  };
  auto next = [&](Stage& g) __attribute__((always_inline)) {
    g.t0 += kWgStep;
    if (g.t0 >= rows) {
      g.t0 = 0;
      g.dy += (int64_t)rows * lda;
    }
  };

  // dY: instruction (wave, p) copies token rows 2*(8*wave + p) and the next;
  // lane l carries slot l % 32 of row l / 32, which holds chunk slot ^ swz(row).
  // Chunks past the last column read the last one: columns are independent,
  // and those are never stored.
  uint32_t dvoff[kDmaPerWave];
#pragma unroll
  for (int p = 0; p < kDmaPerWave; ++p) {
    const int r = 16 * wave + 2 * p + (lane >> 5);
    dvoff[p] = (uint32_t)min(r, rows - 1) * (uint32_t)(lda * 2) +
               min((lane & 31) ^ lds_swizzle_k(r), (it.na - n0) / 8 - 1) * 16;
  }
  auto dy_base = [&](const Stage& g) __attribute__((always_inline)) {
    return g.dy + min(g.t0, last_base) * lda + n0;
  };
  auto copy_dy = [&](const u16* base, int buf, int p) __attribute__((always_inline)) {
    dma16s(base, dvoff[p], lds0 + buf * kStageBytes + (wave * kDmaPerWave + p) * 1024);
  };
  // X: chunk c of a thread is bytes 16*(tid % 16) .. of token row 16c + tid/16.
  const int qr = tid >> 4, qc = tid & 15;
  const int qcol = k0 + 16 * min(qc, (it.k - 1 - k0) / 16);  // the last chunk with a column of this matrix
  uint32_t qvoff[kChunks], evoff[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const uint32_t r = (uint32_t)min(16 * c + qr, rows - 1);
    qvoff[c] = r * (uint32_t)ldq + qcol;
    evoff[c] = r * (uint32_t)lde + qcol / kGroup;
  }
  // Two sets of registers: one is decoded while the next stage's bytes arrive
  // in the other.
  u32x4 qv[2][kChunks];
  uint32_t ev[2][kChunks];
  auto load_x = [&](const Stage& g, int set, int c) __attribute__((always_inline)) {
    const int64_t t = min(g.t0, last_base);
    qv[set][c] = gload16(xq + t * ldq + qvoff[c]);
    ev[set][c] = *((const g_u8*)(xe + t * lde + evoff[c]));
  };
  // Bytes 4w .. 4w+3 of chunk c as bf16; w odd completes 16 bytes, which are
  // stored. Rows that are not the stage's become zeros.
  const uint32_t xoff = kOpBytes + qr * kRowBytes, xslot = (uint32_t)(2 * qc) ^ lds_swizzle_k(qr);
  u32x4 half;
  auto write_x = [&](int skip, int set, int buf, int c, int w) __attribute__((always_inline)) {
    const int r = 16 * c + qr;
    const bool live = r >= skip && r < rows;
    float v[4];
    q8_decode4(live ? qv[set][c][w] : 0u, live ? q8_unit(ev[set][c]) : 0.f, KIND, v);
    half[2 * (w & 1)] = pack_bf16x2(v[0], v[1]);
    half[2 * (w & 1) + 1] = pack_bf16x2(v[2], v[3]);
    if (w & 1)
      *reinterpret_cast<u32x4*>(smem + buf * kStageBytes + xoff + 16 * c * kRowBytes + ((xslot ^ (w >> 1)) << 4)) = half;
  };
  // The same for dY, once it is in LDS.
  auto clear_dy = [&](const Stage& g, int buf) __attribute__((always_inline)) {
    const int skip = g.t0 - min(g.t0, last_base);
    if (skip == 0 && rows >= kWgStep) return;
    const u32x4 z = {0u, 0u, 0u, 0u};
    for (int o = tid * 16; o < kOpBytes; o += 256 * 16) {
      const int r = o / kRowBytes;
      if (r < skip || r >= rows) *reinterpret_cast<u32x4*>(smem + buf * kStageBytes + o) = z;
    }
    __syncthreads();
  };

  // Fragments: lane group G = lane/16, lane i16 points at token row 8*(G/2) +
  // i16/4 (+4 for the upper half, +16 per sub-step) and four columns.
  const int G = lane >> 4, i16 = lane & 15;
  const uint32_t frow = (8 * (G >> 1) + (i16 >> 2)) * kRowBytes;
  uint32_t foff[2][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int col = 32 * j + 16 * (G & 1) + 4 * (i16 & 3);
    foff[0][j] = frow + ((((wm * 128 + col) >> 3) ^ lds_swizzle_k(i16 >> 2)) << 4) + 8 * (i16 & 1);
    foff[1][j] = kOpBytes + frow + ((((wn * 128 + col) >> 3) ^ lds_swizzle_k(i16 >> 2)) << 4) + 8 * (i16 & 1);
  }
  bf16x8 fy[2][4], fx[2][4];
  // Fragment f of a sub-step, in the order in which the MFMAs need them:
  // dY block 0, X blocks 0 .. 3, dY blocks 1 .. 3.
  auto read_frag = [&](int b, int buf, int kk, int f) __attribute__((always_inline)) {
    const bool is_x = f >= 1 && f <= 4;
    const int j = is_x ? f - 1 : f == 0 ? 0 : f - 4;
    const unsigned char* p = smem + buf * kStageBytes + kk * 16 * kRowBytes + foff[is_x][j];
    const v4i16 lo = lds_read_tr(p), hi = lds_read_tr(p + 4 * kRowBytes);
    const bf16x8 v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    if (is_x) fx[b][j] = v;
    else fy[b][j] = v;
  };

  // One stage is 64 MFMAs per wave. Between two of them goes a little of
  // everything else, in a fixed order: the fragments of the next sub-step, the
  // copies of the next stage's dY, the loads of the X bytes after that, and
  // the decoding of the next stage's X. The last sub-step's fragments are in
  // registers halfway through it: there the workgroup meets, and the next
  // stage's first fragments are read under the remaining MFMAs.
  auto stage = [&](int s, Stage& gd, Stage& gx) __attribute__((always_inline)) {
    const int P = (s - s_begin) & 1;
    if (s + 1 < s_end) next(gd);
    if (s + 2 < s_end) next(gx);
    const u16* base = dy_base(gd);
    const int skip = gd.t0 - min(gd.t0, last_base);
    // The next stage's X bytes have arrived (the last wait was for
    // everything). Naming them here places the compiler's own wait for them
    // before the copies of dY, which it would otherwise wait for too.
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      qv[0][c] = qv[1][c];
      ev[0][c] = ev[1][c];
      asm volatile("" : "+v"(qv[0][c]), "+v"(ev[0][c]));
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int m = 0; m < 16; ++m) {
        const int slot = 16 * kk + m;
        if (slot == 56) {
          wait_vmcnt<0>();
          __syncthreads();
          clear_dy(gd, P ^ 1);
        }
        acc[m >> 2][m & 3] =
            __builtin_amdgcn_mfma_f32_32x32x16_bf16(fx[kk & 1][m & 3], fy[kk & 1][m >> 2], acc[m >> 2][m & 3], 0, 0, 0);
        if (kk < 3 && m < 8) read_frag((kk + 1) & 1, P, kk + 1, m);
        if (slot >= 56) read_frag(0, P ^ 1, 0, slot - 56);
        if (slot < 16 && m % 2 == 1) copy_dy(base, P ^ 1, m / 2);
        if (slot >= 16 && slot < 24 && m % 2 == 0) load_x(gx, 1, m / 2);
        if (slot >= 3 && slot < 51 && slot % 3 == 0) write_x(skip, 0, P ^ 1, (slot / 3 - 1) / 4, (slot / 3 - 1) % 4);
        __builtin_amdgcn_sched_barrier(0);
      }
  };

  if (s_begin < s_end) {
    const int plane = s_begin / per_plane;
    Stage gd{static_cast<const u16*>(it.dy) + (int64_t)plane * rows * lda, (s_begin - plane * per_plane) * kWgStep};
    Stage gx = gd;  // one stage further: the loads of X run two stages ahead
#pragma unroll
    for (int c = 0; c < kChunks; ++c) load_x(gx, 0, c);
    const u16* base = dy_base(gd);
#pragma unroll
    for (int p = 0; p < kDmaPerWave; ++p) copy_dy(base, 0, p);
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int w = 0; w < 4; ++w) write_x(gd.t0 - min(gd.t0, last_base), 0, 0, c, w);
    if (s_begin + 1 < s_end) next(gx);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) load_x(gx, 1, c);
    wait_vmcnt<0>();
    __syncthreads();
    clear_dy(gd, 0);
#pragma unroll
    for (int f = 0; f < 8; ++f) read_frag(0, 0, 0, f);
    // Steps past the last load a stage again and use nothing of it.
    for (int s = s_begin; s < s_end; ++s) stage(s, gd, gx);
    __syncthreads();  // the last fragments have been read
  }

  // The tile leaves through LDS, in fp32 and in two halves (blocks 0, 1 and
  // 2, 3 of every wave: 128 rows of 256), so that a wave stores whole rows. The 16-byte
  // unit u of row r sits at unit u ^ (r % 64).
  const bool scale_f32 = a->scale_f32, g_f32 = a->g_f32;
  const int ftid = fresh_tid(), flane = ftid & 63;  // keeps these addresses out of the loop's registers
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (half) __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int r = wm * 64 + 32 * i + (flane & 31), u = wn * 32 + 8 * j + 2 * g + (flane >> 5);
          const f32x16& t = acc[2 * half + i][j];
          *reinterpret_cast<f32x4*>(smem + r * 1024 + ((u ^ (r & 63)) << 4)) =
              f32x4{t[4 * g], t[4 * g + 1], t[4 * g + 2], t[4 * g + 3]};
        }
    __syncthreads();
#pragma unroll 4
    for (int q = 0; q < 32; ++q) {
      const int r = 4 * q + wave;
      const f32x4 t = *reinterpret_cast<const f32x4*>(smem + r * 1024 + ((flane ^ (r & 63)) << 4));
      const float v[4] = {t[0], t[1], t[2], t[3]};
      const int n = (r >> 6) * 128 + half * 64 + (r & 63);
      if (it.splits > 1)
        Vec4<float>::store(a->partial + (int64_t)(it.part0 + local) * kWgPart + n * kWgTile + flane * 4, v);
      else
        store_grad(it, scale_f32, g_f32, n0 + n, k0 + flane * 4, v);
    }
  }
}

// Adds an item's partial tiles in split order and stores the gradient. A
// workgroup takes four rows of one tile: 64 workgroups per tile.
__global__ void __launch_bounds__(256) wgrad_reduce_kernel(WgArgs) {
  const ArgsPtr a = (ArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
  // workgroups are numbered over the tiles of the items with splits
  int b = blockIdx.x, idx = 0;
  for (; idx < a->n_items; ++idx) {
    const int mine = a->item[idx].splits > 1 ? a->item[idx].tiles_n * a->item[idx].tiles_k * 64 : 0;
    if (b < mine) break;
    b -= mine;
  }
  const __attribute__((address_space(4))) WgItem& it = a->item[idx];
  const int tiles = it.tiles_n * it.tiles_k, tile = b >> 6;
  const int f = (b & 63) * 256 + threadIdx.x;
  const float* p = a->partial + (int64_t)(it.part0 + tile) * kWgPart + f * 4;
  float v[4];
  Vec4<float>::load(p, v);
  for (int s = 1; s < it.splits; ++s) {
    float w[4];
    Vec4<float>::load(p + (int64_t)s * tiles * kWgPart, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += w[i];
  }
  int tn, tk;
  tile_of(tile, it.tiles_n, it.tiles_k, tn, tk);
  store_grad(it, a->scale_f32, a->g_f32, tn * kWgTile + f / 64, tk * kWgTile + f % 64 * 4, v);
}

hipError_t launch_wgrad(const WgArgs& args, int kind, hipStream_t s) {
  if (args.units > 0) {
    if (kind == MUON_Q8_INT8) hipLaunchKernelGGL(wgrad_kernel<MUON_Q8_INT8>, dim3(args.units), dim3(256), 0, s, args);
    else hipLaunchKernelGGL(wgrad_kernel<MUON_Q8_E4M3>, dim3(args.units), dim3(256), 0, s, args);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  int64_t blocks = 0;
  for (int i = 0; i < args.n_items; ++i)
    if (args.item[i].splits > 1) blocks += (int64_t)args.item[i].tiles_n * args.item[i].tiles_k * 64;
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL(wgrad_reduce_kernel, dim3((uint32_t)blocks), dim3(256), 0, s, args);
  return hipGetLastError();
}

// dY in other layouts than the product's (fp32, unaligned rows, a width that is
// no multiple of 8): rewritten once, as one bf16 plane or as the three planes
// lo, mid, hi of fp32 values, rows of lda columns (zeros past n). hi is x
// rounded toward zero to bf16, mid and lo the same of what is left: 8 bits
// each, exact for the 24 bits of a normal fp32 number, and never past the
// largest finite value. Infinities and NaNs stay in hi alone.
template <class T, int PARTS>
__global__ void __launch_bounds__(256) wgrad_pack_kernel(const T* dy, int64_t ld, u16* out, int32_t rows, int32_t n,
                                                         int64_t lda) {
  const int64_t octets = lda / 8, count = octets * rows;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / octets, c0 = (i - row * octets) * 8;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c0 + e < n ? Elem<T>::load(dy + row * ld + c0 + e) : 0.f;
    u16* o = out + row * lda + c0;
    if constexpr (PARTS == 1) {
      u32x4 t;
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
      *((g_u32x4*)o) = t;
    } else {
      u32x4 t[3];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t b[3][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float x = v[2 * e + h];
          const uint32_t bits = __float_as_uint(x);
          const bool fine = (bits & 0x7f800000u) != 0x7f800000u;
          b[2][h] = fine ? bits & 0xffff0000u : __float_as_uint(bf16_to_f32(f32_to_bf16(x)));
          const float r = fine ? x - __uint_as_float(b[2][h]) : 0.f;
          b[1][h] = __float_as_uint(r) & 0xffff0000u;
          b[0][h] = __float_as_uint(r - __uint_as_float(b[1][h])) & 0xffff0000u;
        }
#pragma unroll
        for (int p = 0; p < 3; ++p) t[p][e] = (b[p][0] >> 16) | b[p][1];
      }
#pragma unroll
      for (int p = 0; p < 3; ++p) *((g_u32x4*)(o + (int64_t)p * rows * lda)) = t[p];
    }
  }
}

hipError_t launch_wgrad_pack(const void* dy, int64_t ld, int dtype, void* out, int32_t rows, int32_t n, int64_t lda,
                             hipStream_t s) {
  const int64_t count = lda / 8 * rows;
  if (count == 0) return hipSuccess;
  const dim3 grid((uint32_t)std::min<int64_t>((count + 255) / 256, 8192));
  if (dtype == MUON_BF16)
    hipLaunchKernelGGL((wgrad_pack_kernel<u16, 1>), grid, dim3(256), 0, s, static_cast<const u16*>(dy), ld,
                       static_cast<u16*>(out), rows, n, lda);
  else
    hipLaunchKernelGGL((wgrad_pack_kernel<float, 3>), grid, dim3(256), 0, s, static_cast<const float*>(dy), ld,
                       static_cast<u16*>(out), rows, n, lda);
  return hipGetLastError();
}

}  // namespace muon
