// gfx950 kernels of 8-bit activation checkpoints and of the norm sites between
// blocks. Up to 8192 columns (backward: 6144) they are bound by HBM: each tensor
// is read once and written once, sums are fp32, and every thread owns 8
// consecutive columns (16 bytes of bf16, 8 bytes of a checkpoint), so a wave
// instruction moves whole lines. Wider rows are right but slow; each kernel says
// what it does with them.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.h"
#include "layer_internal.h"
#include "q8.h"

namespace muon {

// ------------------------------------------------------------ eight columns

// Columns c0 .. c0+7 of a row, as they lie in memory: rows that are loaded
// ahead, and weights that stay in registers, take half the space so. Columns at
// or past cols are 0 once widened, and are not written. VEC: the row is 16-byte
// aligned and cols a multiple of 8; otherwise only a row's last columns are
// loaded one by one, at clamped addresses, and nothing is done to what was
// loaded until it is widened, so that no load waits for another.
template <class T>
struct Raw8 {
  u32x4 w[sizeof(T) / 2];
};

template <class T, bool VEC>
MUON_INLINE Raw8<T> load_raw(const T* row, int64_t c0, int64_t cols) {
  constexpr int N = sizeof(T) / 2, PER = 16 / sizeof(T);
  Raw8<T> r;
#pragma unroll
  for (int h = 0; h < N; ++h) r.w[h] = u32x4{0u, 0u, 0u, 0u};
  if (VEC ? c0 < cols : c0 + 8 <= cols) {
#pragma unroll
    for (int h = 0; h < N; ++h) r.w[h] = VEC ? gload16(row + c0 + h * PER) : gload16_any(row + c0 + h * PER);
  } else if (!VEC && c0 < cols) {
    typedef T Tx8 __attribute__((ext_vector_type(8)));
    Tx8 t;
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = *((const T __attribute__((address_space(1)))*)(row + min(c0 + i, cols - 1)));
    r = __builtin_bit_cast(Raw8<T>, t);
  }
  return r;
}

template <class T, bool VEC>
MUON_INLINE void widen(const Raw8<T>& r, int64_t c0, int64_t cols, float v[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(r.w[i >> 2][i & 3]);
    else v[i] = __uint_as_float(i & 1 ? r.w[0][i >> 1] & 0xffff0000u : r.w[0][i >> 1] << 16);
    if (!VEC) v[i] = c0 + i < cols ? v[i] : 0.f;
  }
}

template <class T, bool VEC>
MUON_INLINE void store8(T* row, int64_t c0, int64_t cols, const float v[8]) {
  constexpr int N = sizeof(T) / 2, PER = 16 / sizeof(T);
  if (VEC ? c0 < cols : c0 + 8 <= cols) {
#pragma unroll
    for (int h = 0; h < N; ++h) {
      u32x4 t;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2) t[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        else t[i] = __float_as_uint(v[4 * h + i]);
      }
      if (VEC) *((g_u32x4*)(row + c0 + h * PER)) = t;
      else gstore16_any(row + c0 + h * PER, t);
    }
  } else if (!VEC) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c0 + i < cols) Elem<T>::store(row + c0 + i, v[i]);
  }
}

// Quantises columns c0 .. c0+7 of one row (4 adjacent lanes hold a group; all
// of them must be here) and stores them. Rows of q are 16-byte aligned and
// padded, so the 8 bytes are always one store.
MUON_INLINE void store_q8(uint8_t* q, uint8_t* e, int64_t c0, int64_t cols, const float v[8], int kind) {
  u32x2 w;
  const uint32_t E = q8_encode(v, kind, w);
  if (c0 >= cols) return;
  *((g_u32x2*)(q + c0)) = w;
  if (c0 % kGroup == 0) *((g_u8*)(e + c0 / kGroup)) = (uint8_t)E;
}

struct RawQ8 {
  u32x2 w;
  uint32_t e;
};

MUON_INLINE RawQ8 load_raw_q8(const muon_q8& p, int64_t row, int64_t c0) {
  RawQ8 r{{0u, 0u}, 127u};
  if (c0 < p.cols) {
    r.w = *((const g_u32x2*)(static_cast<const uint8_t*>(p.q) + row * p.ldq + c0));
    r.e = *((const g_u8*)(static_cast<const uint8_t*>(p.e) + row * p.lde + c0 / kGroup));
  }
  return r;
}

template <bool VEC>
MUON_INLINE void widen_q8(const RawQ8& r, int64_t c0, int64_t cols, int kind, float v[8]) {
  q8_decode(r.w, r.e, kind, v);
  if constexpr (!VEC) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c0 + i < cols ? v[i] : 0.f;  // padding bytes are not the row's
  }
}

// ------------------------------------------------------------ save and load

// A workgroup is tx lanes wide (8 columns each) and 256/tx rows tall; tx is a
// power of two >= 4, so a group's four lanes are neighbours. A thread takes two
// rows, all loads before the first store: 4096 x 25600 bf16 saved and loaded in
// 131 us, 4.9 TB/s, which is what a copy reaches (one row 139 us, four 133,
// eight 134).
constexpr int kQ8Rows = 2;
struct Q8Args {
  void* x;
  int64_t ldx;
  muon_q8 p;
  int32_t log_tx;
};

template <class T, bool VEC, bool SAVE>
__global__ void __launch_bounds__(256) q8_kernel(Q8Args a) {
  const int tx = 1 << a.log_tx, ty = 256 >> a.log_tx;
  const int64_t c0 = ((int64_t)blockIdx.y * tx + (threadIdx.x & (tx - 1))) * 8;
  const int64_t cols = a.p.cols, rows = a.p.rows;
  for (int64_t row0 = (int64_t)blockIdx.x * ty * kQ8Rows + (threadIdx.x >> a.log_tx); row0 < rows;
       row0 += (int64_t)gridDim.x * ty * kQ8Rows) {
    Raw8<T> x[kQ8Rows];
    RawQ8 q[kQ8Rows];
#pragma unroll
    for (int u = 0; u < kQ8Rows; ++u) {
      const int64_t row = row0 + u * ty;
      if (row >= rows) break;
      if constexpr (SAVE) x[u] = load_raw<T, VEC>(static_cast<const T*>(a.x) + row * a.ldx, c0, cols);
      else q[u] = load_raw_q8(a.p, row, c0);
    }
#pragma unroll
    for (int u = 0; u < kQ8Rows; ++u) {
      const int64_t row = row0 + u * ty;
      if (row >= rows) break;
      float v[8];
      if constexpr (SAVE) {
        widen<T, VEC>(x[u], c0, cols, v);
        store_q8(static_cast<uint8_t*>(a.p.q) + row * a.p.ldq, static_cast<uint8_t*>(a.p.e) + row * a.p.lde, c0, cols, v,
                 a.p.kind);
      } else {
        widen_q8<VEC>(q[u], c0, cols, a.p.kind, v);
        store8<T, VEC>(static_cast<T*>(a.x) + row * a.ldx, c0, cols, v);
      }
    }
  }
}

static bool rows_aligned(const void* p, int64_t ld, int elem) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * elem % 16 == 0;
}

template <bool SAVE>
static hipError_t launch_q8(const void* x, int64_t ldx, int dtype, const muon_q8& p, hipStream_t s) {
  if (p.rows == 0) return hipSuccess;
  const int64_t octets = (p.cols + kGroup - 1) / kGroup * 4;
  Q8Args a{const_cast<void*>(x), ldx, p, 2};
  while (a.log_tx < 8 && (int64_t(1) << a.log_tx) < octets) ++a.log_tx;
  const int64_t gy = (octets + (1 << a.log_tx) - 1) >> a.log_tx;  // at most 2^24 / 2048
  const int64_t per = (256 >> a.log_tx) * kQ8Rows, gx = (p.rows + per - 1) / per;
  const dim3 grid((uint32_t)std::min<int64_t>(gx, std::max<int64_t>(1, (1 << 20) / gy)), (uint32_t)gy);
  const int elem = dtype == MUON_BF16 ? 2 : 4;
  const bool vec = p.cols % 8 == 0 && rows_aligned(x, ldx, elem);
  if (dtype == MUON_BF16) {
    if (vec) hipLaunchKernelGGL((q8_kernel<u16, true, SAVE>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((q8_kernel<u16, false, SAVE>), grid, dim3(256), 0, s, a);
  } else {
    if (vec) hipLaunchKernelGGL((q8_kernel<float, true, SAVE>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((q8_kernel<float, false, SAVE>), grid, dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

hipError_t launch_q8_save(const void* x, int64_t ldx, int dtype, const muon_q8& out, hipStream_t s) {
  return launch_q8<true>(x, ldx, dtype, out, s);
}
hipError_t launch_q8_load(const muon_q8& in, void* x, int64_t ldx, int dtype, hipStream_t s) {
  return launch_q8<false>(x, ldx, dtype, in, s);
}

// ------------------------------------------------------------ norm sites

// x plus x of the lane that DPP control C names (0 where it names none).
template <int C, int ROWS = 0xf>
MUON_INLINE float dpp_add(float x) {
  return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), C, ROWS, 0xf, true));
}
// Sums over rows of 16 lanes, in the last lane of each; over the wave, in lane 63.
MUON_INLINE float row16_sum(float x) {
  x = dpp_add<0x111>(x);  // row_shr 1, 2, 4, 8
  x = dpp_add<0x112>(x);
  x = dpp_add<0x114>(x);
  return dpp_add<0x118>(x);
}
MUON_INLINE float wave_sum(float x) {
  x = row16_sum(x);
  x = dpp_add<0x142, 0xa>(x);     // lane 15 of a row to the next, rows 1 and 3
  return dpp_add<0x143, 0xc>(x);  // lane 31 to rows 2 and 3
}
MUON_INLINE float lane_value(float x, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}

// N sums over the workgroup at once, in every thread, in a fixed order. `red`
// holds 16*N floats; two calls in a row need two buffers.
template <int N>
MUON_INLINE void block_sum(float (&v)[N], float* red) {
  const int waves = blockDim.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (waves == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane_value(v[i], 63);
    return;
  }
  if (lane == 63) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[16 * i + (threadIdx.x >> 6)] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = (lane & 15) < waves ? red[16 * i + (lane & 15)] : 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane_value(row16_sum(v[i]), 15);
}

// One row per workgroup at a time, or, in rows of one wave, one per wave
// (rows_per of them): thread x holds columns 8x .. 8x+7 (VPT times, blockDim.x
// threads apart). The row stays in registers between its two
// norms, so every tensor moves once. With VPT = 1 there are registers left to
// load the weights once and to have the next row's loads in flight. 4096 x 5120
// bf16: 29 us with its tensors partly in cache, 36 without (4.7 TB/s; a copy
// 4.9); one row 4.1 to 4.8 us, a chain of loads and two sums. 1024 threads have
// 128 registers each, which hold VPT = 2 of aligned bf16 only (1024 x 16384: 35
// us, 3.9 TB/s); other rows past 8192 columns spill 2 to 78 registers, and VPT =
// 4 73 to 386 (512 x 32768 bf16: 63 us, 2.1 TB/s; unaligned 119).
template <class T, int VPT, bool VEC>
__global__ void __launch_bounds__(1024) norm_forward_kernel(muon_norm_site s, int32_t rows_per) {
  __shared__ float red[2][16];
  const int64_t cols = s.cols;
  const float inv_cols = 1.f / (float)cols;
  const bool post = s.w_post != nullptr, per_row = s.gate && s.ld_gate != 0;
  int64_t c0[VPT];
  Raw8<T> b[VPT], r[VPT], gt[VPT], w1[VPT], w2[VPT];
  auto load = [&](int64_t row) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      b[p] = load_raw<T, VEC>(static_cast<const T*>(s.branch) + row * s.ld_branch, c0[p], cols);
      r[p] = load_raw<T, VEC>(static_cast<const T*>(s.residual) + row * s.ld_residual, c0[p], cols);
      if (per_row) gt[p] = load_raw<T, VEC>(static_cast<const T*>(s.gate) + row * s.ld_gate, c0[p], cols);
    }
  };
  auto load_weights = [&](int p) __attribute__((always_inline)) {
    w1[p] = load_raw<T, VEC>(static_cast<const T*>(s.w_pre), c0[p], cols);
    if (post) w2[p] = load_raw<T, VEC>(static_cast<const T*>(s.w_post), c0[p], cols);
    if (s.gate && !per_row) gt[p] = load_raw<T, VEC>(static_cast<const T*>(s.gate), c0[p], cols);
  };
#pragma unroll
  for (int p = 0; p < VPT; ++p) c0[p] = ((int64_t)p * blockDim.x + threadIdx.x) * 8;
  // The same in a whole wave, and said so: row addresses stay in scalar registers.
  // rows_per is blockDim.y, which would take another load to know.
  const int sub = __builtin_amdgcn_readfirstlane(threadIdx.y);
  const int64_t row0 = (int64_t)blockIdx.x * rows_per + sub, step = (int64_t)gridDim.x * rows_per;
  if (row0 >= s.rows) return;  // a wave of its own: nothing waits for it
  if (VPT == 1) {
    load(row0);
    load_weights(0);
  }
  for (int64_t row = row0; row < s.rows; row += step) {
    float v[VPT][8], y[VPT][8], g[VPT][8];
    float sum[1] = {0.f};
    if (VPT > 1) load(row);
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      widen<T, VEC>(b[p], c0[p], cols, v[p]);
      widen<T, VEC>(r[p], c0[p], cols, y[p]);
      if (per_row) widen<T, VEC>(gt[p], c0[p], cols, g[p]);
    }
    if (VPT == 1 && row + step < s.rows) load(row + step);
    if (post || s.rstd_b) {  // without a norm after the block it is only kept
#pragma unroll
      for (int p = 0; p < VPT; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[0] += v[p][i] * v[p][i];
      block_sum(sum, red[0]);
      const float rb = 1.f / sqrtf(sum[0] * inv_cols + s.eps);
      if (threadIdx.x == 0 && s.rstd_b) *((g_f32*)(s.rstd_b + row)) = rb;
      if (post) {
#pragma unroll
        for (int p = 0; p < VPT; ++p)
#pragma unroll
          for (int i = 0; i < 8; ++i) v[p][i] *= rb;
      }
    }
    sum[0] = 0.f;
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      if (VPT > 1) load_weights(p);
      if (s.v.q)
        store_q8(static_cast<uint8_t*>(s.v.q) + row * s.v.ldq, static_cast<uint8_t*>(s.v.e) + row * s.v.lde, c0[p],
                 cols, v[p], s.v.kind);
      float w[8];
      if (post) {
        widen<T, VEC>(w2[p], c0[p], cols, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[p][i] *= w[i];
      }
      if (s.gate) {
        if (!per_row) widen<T, VEC>(gt[p], c0[p], cols, g[p]);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[p][i] *= g[p][i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[p][i] = s.res_scale * y[p][i] + s.branch_scale * v[p][i];
        sum[0] += y[p][i] * y[p][i];
      }
      store8<T, VEC>(static_cast<T*>(s.y) + row * s.ld_y, c0[p], cols, y[p]);
    }
    block_sum(sum, red[1]);
    const float ry = 1.f / sqrtf(sum[0] * inv_cols + s.eps);
    if (threadIdx.x == 0 && s.rstd_y) *((g_f32*)(s.rstd_y + row)) = ry;
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[p][i] *= ry;
      if (s.u.q)
        store_q8(static_cast<uint8_t*>(s.u.q) + row * s.u.ldq, static_cast<uint8_t*>(s.u.e) + row * s.u.lde, c0[p],
                 cols, y[p], s.u.kind);
      widen<T, VEC>(w1[p], c0[p], cols, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] *= y[p][i];
      store8<T, VEC>(static_cast<T*>(s.h) + row * s.ld_h, c0[p], cols, w);
    }
    // The next row's first sum writes red[0], which every thread has read
    // before this row's second barrier; without a norm after the block there
    // is only red[1], which would be written while it is still read.
    if (!post && blockDim.x > 64) __syncthreads();
  }
}

// Rows blockIdx.x, + gridDim.x, ... The mean over dv*v needs s, which needs the
// mean over du*u; written out, both follow from three sums that are formed at
// once: with a = branch_scale*gate*w_post,
//   mean(dv*v) = mean(a*v*(dy + rstd_y*du)) - rstd_y * mean(du*u) * mean(a*v*u),
// so a row costs one barrier. Each thread keeps its columns' partial sums of
// the weight gradients in registers and stores them once. With VPT = 1 the row
// stays in registers too, weights are loaded once and loads run a row ahead;
// wider rows are read again (from cache) after their sums. Rows of one wave go
// one to a wave, whose sums are added at the end; a launch of one workgroup
// stores the weight gradients themselves. MAXT: the most threads of a
// workgroup, which sets the registers of each. 16384 x 2048 bf16: 72 to 76 us,
// 4.4 to 4.6 TB/s; 4096 x 5120: 56 to 59 us, 3.6 to 3.8 TB/s, where one workgroup
// of 10 waves is on a CU, its vector units are at work 43% of the time and its
// waves wait for memory 57% of theirs. Reading rows twice costs 6145 to 8192
// columns half of that (4096 x 8192: 119 us, 2.8 TB/s). Past those the sums of a
// thread's 32 columns do not fit its registers and 117 to 556 of them spill: 1024
// x 16384 takes 198 us, 0.85 TB/s. Unaligned rows spill 86 to 90 from 6145
// columns on (2048 x 8191 bf16: 162 us), and in fp32 10 from 4097.
template <class T, int VPT, bool VEC, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_backward_kernel(muon_norm_site s, muon_norm_grads g, int32_t rows_per) {
  __shared__ float red[2][48];
  __shared__ float join[MAXT == 512 && VPT == 1 ? kNormRowsBackward * 512 : 1];
  const int64_t cols = s.cols;
  const float inv_cols = 1.f / (float)cols;
  const bool post = s.w_post != nullptr, per_row = s.gate && s.ld_gate != 0;
  const bool need_v = post || s.gate;
  float acc[3][VPT][8];
#pragma unroll
  for (int w = 0; w < 3; ++w)
#pragma unroll
    for (int p = 0; p < VPT; ++p)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[w][p][i] = 0.f;

  Raw8<T> rdh, rdy, rg, w1, w2;  // of one row's eight columns, as loaded
  RawQ8 ru, rv;
  float ry = 0.f, rb = 1.f;
  auto col0 = [&](int p) { return ((int64_t)p * blockDim.x + threadIdx.x) * 8; };
  auto load = [&](int64_t row, int p) __attribute__((always_inline)) {
    const int64_t c0 = col0(p);
    rdh = load_raw<T, VEC>(static_cast<const T*>(g.dh) + row * g.ld_dh, c0, cols);
    if (g.dy) rdy = load_raw<T, VEC>(static_cast<const T*>(g.dy) + row * g.ld_dy, c0, cols);
    ru = load_raw_q8(s.u, row, c0);
    if (need_v) rv = load_raw_q8(s.v, row, c0);
    if (per_row) rg = load_raw<T, VEC>(static_cast<const T*>(s.gate) + row * s.ld_gate, c0, cols);
    ry = *((const g_f32*)(s.rstd_y + row));
    if (post) rb = *((const g_f32*)(s.rstd_b + row));
  };
  auto load_weights = [&](int p) __attribute__((always_inline)) {
    const int64_t c0 = col0(p);
    w1 = load_raw<T, VEC>(static_cast<const T*>(s.w_pre), c0, cols);
    if (post) w2 = load_raw<T, VEC>(static_cast<const T*>(s.w_post), c0, cols);
    if (s.gate && !per_row) rg = load_raw<T, VEC>(static_cast<const T*>(s.gate), c0, cols);
  };
  // Eight columns of the row: t is dy + rstd_y*du, gt the gate as loaded.
  struct Cols {
    float u[8], v[8], t[8];
    Raw8<T> gt;
    float ry, rb;
  };
  auto widen_row = [&](Cols& c, float dh[8], int p) __attribute__((always_inline)) {
    const int64_t c0 = col0(p);
    widen<T, VEC>(rdh, c0, cols, dh);
#pragma unroll
    for (int i = 0; i < 8; ++i) c.t[i] = c.v[i] = 0.f;
    if (g.dy) widen<T, VEC>(rdy, c0, cols, c.t);
    widen_q8<VEC>(ru, c0, cols, s.u.kind, c.u);
    if (need_v) widen_q8<VEC>(rv, c0, cols, s.v.kind, c.v);
    if (per_row) c.gt = rg;
    c.ry = ry, c.rb = rb;
  };
  auto gate_of = [&](const Cols& c, int p, float gt[8]) __attribute__((always_inline)) {
    if (s.gate) {
      widen<T, VEC>(per_row ? c.gt : rg, col0(p), cols, gt);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) gt[i] = 1.f;
    }
  };
  // The row's share of its three sums.
  auto add_sums = [&](Cols& c, int p, const float dh[8], float (&sum)[3]) __attribute__((always_inline)) {
    float w[8];
    widen<T, VEC>(w1, col0(p), cols, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float du = dh[i] * w[i];
      sum[0] += du * c.u[i];
      c.t[i] += c.ry * du;
    }
    if (post) {
      float gt[8];
      widen<T, VEC>(w2, col0(p), cols, w);
      gate_of(c, p, gt);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float av = gt[i] * w[i] * c.v[i];
        sum[1] += av * c.t[i];
        sum[2] += av * c.u[i];
      }
    }
  };
  auto finish = [&](Cols& c, int64_t row, int p, const float (&sum)[3]) __attribute__((always_inline)) {
    const int64_t c0 = col0(p);
    const float c1 = c.ry * (sum[0] * inv_cols);
    const float c2 = s.branch_scale * (sum[1] - c1 * sum[2]) * inv_cols;
    float o[8], w[8], gt[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c.t[i] -= c1 * c.u[i];  // s
      o[i] = s.res_scale * c.t[i];
      c.t[i] *= s.branch_scale;
    }
    store8<T, VEC>(static_cast<T*>(g.d_residual) + row * g.ld_d_residual, c0, cols, o);
    if (post) {
      widen<T, VEC>(w2, col0(p), cols, w);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 1.f;
    }
    gate_of(c, p, gt);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      o[i] = c.t[i] * w[i] * c.v[i];
      acc[2][p][i] += o[i];
      c.t[i] *= gt[i];
      acc[1][p][i] += c.t[i] * c.v[i];
    }
    if (per_row && g.d_gate) store8<T, VEC>(static_cast<T*>(g.d_gate) + row * g.ld_d_gate, c0, cols, o);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = post ? c.rb * (c.t[i] * w[i] - c.v[i] * c2) : c.t[i];
    store8<T, VEC>(static_cast<T*>(g.d_branch) + row * g.ld_d_branch, c0, cols, o);
  };

  const int y = __builtin_amdgcn_readfirstlane(threadIdx.y);
  const int64_t row0 = (int64_t)blockIdx.x * rows_per + y, step = (int64_t)gridDim.x * rows_per;
  if (VPT == 1 && row0 < s.rows) {
    load(row0, 0);
    load_weights(0);
  }
  int flip = 0;
  for (int64_t row = row0; row < s.rows; row += step, flip ^= 1) {
    float sum[3] = {0.f, 0.f, 0.f};
    Cols c;
    float dh[8];
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      if (VPT > 1) {
        load(row, p);
        load_weights(p);
      }
      widen_row(c, dh, p);
      if (VPT == 1 && row + step < s.rows) load(row + step, 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[0][p][i] += dh[i] * c.u[i];
      add_sums(c, p, dh, sum);
      if (VPT > 1) __builtin_amdgcn_sched_barrier(0);  // eight columns' registers at a time
    }
    block_sum(sum, red[flip]);
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      if (VPT > 1) {
        float none[3] = {0.f, 0.f, 0.f};
        load(row, p);
        load_weights(p);
        widen_row(c, dh, p);
        add_sums(c, p, dh, none);
      }
      finish(c, row, p, sum);
      if (VPT > 1) __builtin_amdgcn_sched_barrier(0);
    }
  }
  if constexpr (MAXT == 512 && VPT == 1) {
    if (rows_per > 1) {
#pragma unroll
      for (int w = 0; w < 3; ++w) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) join[y * 512 + threadIdx.x * 8 + i] = acc[w][0][i];
        __syncthreads();
        if (y == 0) {
          for (int o = 1; o < rows_per; ++o)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[w][0][i] += join[o * 512 + threadIdx.x * 8 + i];
        }
      }
      if (y != 0) return;
    }
  }
  if (gridDim.x == 1) {
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      if (g.d_w_pre) store8<T, VEC>(static_cast<T*>(g.d_w_pre), col0(p), cols, acc[0][p]);
      if (g.d_w_post) store8<T, VEC>(static_cast<T*>(g.d_w_post), col0(p), cols, acc[1][p]);
      if (g.d_gate && !per_row) store8<T, VEC>(static_cast<T*>(g.d_gate), col0(p), cols, acc[2][p]);
    }
    return;
  }
  const int64_t pitch = (cols + 7) / 8 * 8;
  float* part = static_cast<float*>(g.workspace) + (int64_t)blockIdx.x * 3 * pitch;
#pragma unroll
  for (int w = 0; w < 3; ++w)
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      if (col0(p) >= cols) continue;
      Vec4<float>::store(part + w * pitch + col0(p), acc[w][p]);
      Vec4<float>::store(part + w * pitch + col0(p) + 4, acc[w][p] + 4);
    }
}

// The weight gradients from the partial sums: 64 columns per workgroup, 16
// waves that each add every 16th partial, joined in order. Three weights of 2048
// columns from 768 workgroups: 4.8 us (15.8 with one load in flight).
template <class T>
__global__ void __launch_bounds__(1024) norm_weights_kernel(const float* part, int32_t blocks, int64_t cols, T* d0,
                                                            T* d1, T* d2) {
  __shared__ float red[16][64];
  T* out = blockIdx.y == 0 ? d0 : blockIdx.y == 1 ? d1 : d2;
  if (!out) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane, pitch = (cols + 7) / 8 * 8;
  float sum = 0.f;
  if (c < cols) {
    const float* p = part + blockIdx.y * pitch + c;
    int b = wave;
    for (; b + 16 * 7 < blocks; b += 16 * 8) {  // eight loads in flight
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = *((const g_f32*)(p + (int64_t)(b + 16 * i) * 3 * pitch));
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += t[i];
    }
    for (; b < blocks; b += 16) sum += *((const g_f32*)(p + (int64_t)b * 3 * pitch));
  }
  red[wave][lane] = sum;
  __syncthreads();
  if (wave != 0 || c >= cols) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) sum += red[w][lane];
  Elem<T>::store(out + c, sum);
}

template <class T>
static hipError_t norm_forward(const muon_norm_site& s, hipStream_t st) {
  if (s.rows == 0) return hipSuccess;
  const int elem = sizeof(T);
  const bool vec = s.cols % 8 == 0 && rows_aligned(s.branch, s.ld_branch, elem) &&
                   rows_aligned(s.residual, s.ld_residual, elem) && rows_aligned(s.y, s.ld_y, elem) &&
                   rows_aligned(s.h, s.ld_h, elem) && rows_aligned(s.w_pre, 0, elem) &&
                   rows_aligned(s.w_post, 0, elem) && rows_aligned(s.gate, s.ld_gate, elem);
  const NormLaunch l = norm_forward_launch(s.rows, s.cols);
  const int vpt = l.vecs;
  const dim3 grid(l.blocks), block(l.threads, l.rows_per);
#define MUON_NORM_F(V, A) hipLaunchKernelGGL((norm_forward_kernel<T, V, A>), grid, block, 0, st, s, l.rows_per)
  if (vec) { if (vpt == 1) MUON_NORM_F(1, true); else if (vpt == 2) MUON_NORM_F(2, true); else MUON_NORM_F(4, true); }
  else { if (vpt == 1) MUON_NORM_F(1, false); else if (vpt == 2) MUON_NORM_F(2, false); else MUON_NORM_F(4, false); }
#undef MUON_NORM_F
  return hipGetLastError();
}

template <class T>
static hipError_t norm_backward(const muon_norm_site& s, const muon_norm_grads& g, hipStream_t st) {
  const int elem = sizeof(T);
  const bool per_row = s.gate && s.ld_gate != 0;
  const bool vec = s.cols % 8 == 0 && rows_aligned(g.dy, g.ld_dy, elem) && rows_aligned(g.dh, g.ld_dh, elem) &&
                   rows_aligned(g.d_residual, g.ld_d_residual, elem) &&
                   rows_aligned(g.d_branch, g.ld_d_branch, elem) && rows_aligned(s.w_pre, 0, elem) &&
                   rows_aligned(s.w_post, 0, elem) && rows_aligned(s.gate, s.ld_gate, elem) &&
                   rows_aligned(g.d_gate, per_row ? g.ld_d_gate : 0, elem) && rows_aligned(g.d_w_pre, 0, elem) &&
                   rows_aligned(g.d_w_post, 0, elem);
  const NormLaunch l = norm_backward_launch(s.rows, s.cols);
  const int vpt = l.vecs;
  if (l.blocks > 0) {
    const dim3 grid(l.blocks), block(l.threads, l.rows_per);
#define MUON_NORM_B(V, M)                                                                                 \
  do {                                                                                                    \
    if (vec) hipLaunchKernelGGL((norm_backward_kernel<T, V, true, M>), grid, block, 0, st, s, g, l.rows_per);         \
    else hipLaunchKernelGGL((norm_backward_kernel<T, V, false, M>), grid, block, 0, st, s, g, l.rows_per);            \
  } while (0)
    if (vpt == 1 && block.x <= 512) MUON_NORM_B(1, 512);
    else if (vpt == 1) MUON_NORM_B(1, 768);
    else if (vpt == 2) MUON_NORM_B(2, 512);
    else if (block.x <= 512) MUON_NORM_B(4, 512);
    else MUON_NORM_B(4, 1024);
#undef MUON_NORM_B
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || l.blocks == 1) return e;
  }
  T* dg = per_row ? nullptr : static_cast<T*>(g.d_gate);
  if (!g.d_w_pre && !g.d_w_post && !dg) return hipSuccess;
  hipLaunchKernelGGL(norm_weights_kernel<T>, dim3((uint32_t)((s.cols + 63) / 64), 3), dim3(1024), 0, st,
                     static_cast<const float*>(g.workspace), l.blocks, s.cols, static_cast<T*>(g.d_w_pre),
                     static_cast<T*>(g.d_w_post), dg);
  return hipGetLastError();
}

hipError_t launch_norm_forward(const muon_norm_site& s, hipStream_t st) {
  return s.dtype == MUON_BF16 ? norm_forward<u16>(s, st) : norm_forward<float>(s, st);
}
hipError_t launch_norm_backward(const muon_norm_site& s, const muon_norm_grads& g, hipStream_t st) {
  return s.dtype == MUON_BF16 ? norm_backward<u16>(s, g, st) : norm_backward<float>(s, g, st);
}

}  // namespace muon
