// gfx950 kernels of the gated feed-forward block,
//   a = x Wgate^T, b = x Wup^T, s = act(a) * b, y = s Wdown^T,
// and of its backward pass from 8-bit checkpoints of a and b,
//   ds = dy Wdown, da = ds * b * act'(a), db = ds * act(a), dx = da Wgate + db Wup.
//
// Four products, each one launch: the two projections side by side in one tile, so
// that the activation, the product and the checkpoints of a, b and s are its
// epilogue; the down projection; ds, whose epilogue makes da and db; and dx, one sum
// over both pairs. The weights are read as they lie: forward along their rows,
// backward with transposing LDS reads.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "product.h"

namespace muon {

// x = hi + mid + lo, each the rest rounded toward zero to bf16 (24 bits of numbers
// of at least 2^-110). Infinities and NaNs stay in hi alone.
MUON_INLINE void cut3(float x, float& hi, float& mid, float& lo) {
  const uint32_t bits = __float_as_uint(x);
  const bool fine = (bits & 0x7f800000u) != 0x7f800000u;
  hi = fine ? __uint_as_float(bits & 0xffff0000u) : x;
  const float r = fine ? x - hi : 0.f;
  mid = __uint_as_float(__float_as_uint(r) & 0xffff0000u);
  lo = __uint_as_float(__float_as_uint(r - mid) & 0xffff0000u);
}

// 1 / (1 + e^-x); e^-x in the hardware's exponential of base 2: a relative error of
// (|x| + 2) 2^-24 or so.
MUON_INLINE float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * x)); }

// act(a) and act'(a).
MUON_INLINE void activation(float a, int act, float& f, float& df) {
  if (act == MUON_ACT_SILU) {
    const float s = sigmoid(a);
    f = a * s;
    df = fmaf(f, 1.f - s, s);
  } else if (act == MUON_ACT_GELU) {
    const float phi = 0.5f + 0.5f * erff(a * 0.70710678f);
    f = a * phi;
    df = fmaf(a * 0.39894228f, __builtin_amdgcn_exp2f(-0.72134752f * a * a), phi);
  } else if (act == MUON_ACT_GELU_TANH) {
    // (1 + tanh u) / 2 = sigmoid(2 u); from |a| = 100 on it is 0 or 1 whatever a^2 is
    const float a2 = fminf(a * a, 1e4f), s = sigmoid(1.5957691216f * a * fmaf(0.044715f, a2, 1.f));
    f = a * s;
    df = fmaf(f * (1.f - s), 1.5957691216f * fmaf(0.134145f, a2, 1.f), s);
  } else {
    f = a > 0.f ? a : a == a ? 0.f : a;
    df = a > 0.f ? 1.f : 0.f;
  }
}

// The bytes and the exponent of eight columns, four lanes a group, into a
// checkpoint. Padding columns (up to a multiple of 16) get 0.
MUON_INLINE void save_run(const __attribute__((address_space(4))) muon_q8& q, int row, int col, bool there, const float v[8]) {
  u32x2 w;
  const uint32_t E = q8_encode(v, q.kind, w);
  if (there && col < ((int)q.cols + 15) / 16 * 16)
    *((g_u32x2*)(static_cast<uint8_t*>(q.q) + (int64_t)row * q.ldq + col)) = w;
  if (there && (col & (kGroup - 1)) == 0 && col < q.cols)
    *((g_u8*)(static_cast<uint8_t*>(q.e) + (int64_t)row * q.lde + col / kGroup)) = (uint8_t)E;
}

// Eight columns as an operand of the next product: bf16, or three planes.
template <class M>
MUON_INLINE void put_planes(const M& mlp, u16* base, int parts, int row, int col, const float v[8]) {
  u16* p = base + (int64_t)row * mlp.ldp + col;
  if (parts == 1) {
    *((g_u32x4*)p) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    return;
  }
  float t[3][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) cut3(v[i], t[2][i], t[1][i], t[0][i]);
#pragma unroll
  for (int q = 0; q < 3; ++q)
    *((g_u32x4*)(p + q * mlp.pp)) =
        u32x4{pack_bf16x2(t[q][0], t[q][1]), pack_bf16x2(t[q][2], t[q][3]), pack_bf16x2(t[q][4], t[q][5]), pack_bf16x2(t[q][6], t[q][7])};
}

// a and b of eight columns: s for the down projection, and the checkpoints. Lanes
// past the last column take part in their group with zeros.
struct PrGateOut {
  static constexpr int OPS = 2;
  PrItemRef it;
  const __attribute__((address_space(4))) PrMlp& mlp;
  int parts;
  MUON_INLINE PrGateOut(PrItemRef item, PrArgsPtr a) : it(item), mlp(a->mlp), parts(a->parts) {}
  MUON_INLINE void emit(int row, int col, float a[8], float b[8]) const {
    const bool there = row < it.m;
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f, df;
      activation(a[i], mlp.act, f, df);
      s[i] = f * b[i];
      if (col + i >= it.n) a[i] = b[i] = s[i] = 0.f;
    }
    if (there && col < it.n) put_planes(mlp, mlp.plane[0], parts, row, col, s);
    if (mlp.a.q) save_run(mlp.a, row, col, there, a);
    if (mlp.b.q) save_run(mlp.b, row, col, there, b);
    if (mlp.s.q) save_run(mlp.s, row, col, there, s);
  }
};

// ds of eight columns, with a and b from their checkpoints.
struct PrGateGradOut {
  static constexpr int OPS = 1;
  PrItemRef it;
  const __attribute__((address_space(4))) PrMlp& mlp;
  int parts;
  bool f32;
  MUON_INLINE PrGateGradOut(PrItemRef item, PrArgsPtr a) : it(item), mlp(a->mlp), parts(a->parts), f32(a->f32) {}
  MUON_INLINE void load(const __attribute__((address_space(4))) muon_q8& q, int row, int col, float v[8]) const {
    const u32x2 w = *((const g_u32x2*)(static_cast<const uint8_t*>(q.q) + (int64_t)row * q.ldq + col));
    const uint32_t E = *((const g_u8*)(static_cast<const uint8_t*>(q.e) + (int64_t)row * q.lde + col / kGroup));
    q8_decode(w, E, q.kind, v);
  }
  MUON_INLINE void emit(int row, int col, float ds[8], float*) const {
    const int live = row < it.m ? it.n - col : 0;
    if (live <= 0) return;
    float a[8], b[8], da[8], db[8];
    load(mlp.a, row, col, a);
    load(mlp.b, row, col, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f, df;
      activation(a[i], mlp.act, f, df);
      da[i] = i < live ? ds[i] * b[i] * df : 0.f;
      db[i] = i < live ? ds[i] * f : 0.f;
    }
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const float* v = d ? db : da;
      if (f32) store_run(static_cast<float*>(mlp.d[d]) + (int64_t)row * mlp.ldd[d] + col, live, v);
      else store_run(static_cast<u16*>(mlp.d[d]) + (int64_t)row * mlp.ldd[d] + col, live, v);
      if (mlp.plane[d]) put_planes(mlp, mlp.plane[d], parts, row, col, v);
    }
  }
};

template <class Z, class Out>
__global__ void __launch_bounds__(Z::NT, Z::WG) mlp_product_kernel(PrArgs) {
  __shared__ __align__(1024) unsigned char smem[Z::LDS];
  pr_run<Z, Out>(smem);
}

template <class Out>
__global__ void __launch_bounds__(256) mlp_join_kernel(PrArgs, int edge) {
  pr_join_of<Out>(edge);
}

template <int MODE, class Out>
static hipError_t launch_tiles(const PrArgs& args, hipStream_t s) {
  typedef PrCfg<256, 256, 128, 2, MODE, 1> Large;
  typedef PrCfg<128, 128, 128, 2, MODE, 2> Medium;
  typedef PrCfg<64, 64, 128, 4, MODE, 2> Small;
  const dim3 block(256);
  if (args.tile == kPrLarge) hipLaunchKernelGGL((mlp_product_kernel<Large, Out>), dim3(pr_grid<Large>(args)), block, 0, s, args);
  else if (args.tile == kPrMedium) hipLaunchKernelGGL((mlp_product_kernel<Medium, Out>), dim3(pr_grid<Medium>(args)), block, 0, s, args);
  else hipLaunchKernelGGL((mlp_product_kernel<Small, Out>), dim3(pr_grid<Small>(args)), block, 0, s, args);
  const hipError_t e = hipGetLastError();
  const int64_t join = pr_join_blocks(args, Out::OPS == 2);
  if (e != hipSuccess || join == 0) return e;
  hipLaunchKernelGGL(mlp_join_kernel<Out>, dim3((uint32_t)join), dim3(256), 0, s, args, kPrEdge[args.tile]);
  return hipGetLastError();
}

hipError_t launch_mlp(const PrArgs& args, int epilogue, bool transposed_b, hipStream_t s) {
  if (epilogue == kPrGate) return launch_tiles<kNT16, PrGateOut>(args, s);
  if (epilogue == kPrGateGrad) return launch_tiles<kNN16, PrGateGradOut>(args, s);
  return transposed_b ? launch_tiles<kNN16, PrStoreOut>(args, s) : launch_tiles<kNT16, PrStoreOut>(args, s);
}

}  // namespace muon
