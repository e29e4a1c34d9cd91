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
//
// 4096 x 2048 x 6144 bf16, silu, int8 checkpoints: 212, 95 + 15, 143 and 175 + 15 us (973,
// 937, 721 and 1085 TFLOP/s), the second terms joining pieces. The epilogues of the first
// and the third are 17 and 22 of 70 us of a 256 x 256 tile, with the matrix units idle:
// all CUs come to them together and move 43 and 84 MB a round (2.7 and 4.2 TB/s; more
// of a thread's runs at once gained nothing). At 5120 x 25600 the products reach 1075
// and 1014 TFLOP/s.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mlp_math.h"
#include "product.h"

namespace muon {

// A checkpoint as a thread of an epilogue sees it: eight columns, always the same.
struct Saved {
  uint8_t *q, *e;
  int64_t ldq, lde;
  int kind;
  uint32_t off, offe;
  int col, cols, cols16;
  bool first;  // of the four lanes of a group
  MUON_INLINE Saved(const __attribute__((address_space(4))) muon_q8& s, PrLane at)
      : q(static_cast<uint8_t*>(pinned(s.q))), e(static_cast<uint8_t*>(pinned(s.e))), ldq(pinned(s.ldq)), lde(pinned(s.lde)),
        kind(pinned(s.kind)) {
    off = (uint32_t)at.row * (uint32_t)ldq + (uint32_t)at.col;
    offe = (uint32_t)at.row * (uint32_t)lde + (uint32_t)(at.col / kGroup);
    col = at.col;
    cols = (int)s.cols;
    cols16 = (cols + 15) / 16 * 16;
    first = (col & (kGroup - 1)) == 0;
  }
  // Columns of a group are four lanes. Padding columns (up to a multiple of 16) get 0.
  // Nontemporal: the next launch reads s as its operand, the backward pass these (a
  // training step of 4096 x 2048 x 6144 1008 -> 1000 us; da and db, which are read at
  // once, 1004 with them too).
  template <class V>
  MUON_INLINE void save(int row, bool there, const float v[8]) const {
    u32x2 w;
    const uint32_t E = q8_encode(v, V::FULL ? V::B : kind, w);
    uint8_t *pq = q + (int64_t)row * ldq, *pe = e + (int64_t)row * lde;
    if (V::FULL || (there && col < cols16)) __builtin_nontemporal_store(w, (g_u32x2*)(pq + off));
    if (first && (V::FULL || (there && col < cols))) *((g_u8*)(pe + offe)) = (uint8_t)E;
  }
  MUON_INLINE void load(int row, u32x2& w, uint32_t& E) const {
    const uint8_t *pq = q + (int64_t)row * ldq, *pe = e + (int64_t)row * lde;
    w = *((const g_u32x2*)(pq + off));
    E = *((const g_u8*)(pe + offe));
  }
};

// Eight columns as an operand of the next product: bf16, or three planes.
struct Planes {
  char* p;
  int64_t ld, plane;  // bytes
  uint32_t off;
  int parts;
  MUON_INLINE Planes(uint16_t* base, const __attribute__((address_space(4))) PrMlp& m, int parts_, PrLane at)
      : p(reinterpret_cast<char*>(pinned(base))), ld(2 * pinned(m.ldp)), plane(2 * pinned(m.pp)), parts(parts_) {
    off = (uint32_t)at.row * (uint32_t)ld + 2u * (uint32_t)at.col;
  }
  template <class V>
  MUON_INLINE void put(int row, const float v[8]) const {
    char* base = p + (int64_t)row * ld;
    if (V::FULL || parts == 1) {
      *((g_u32x4*)(base + off)) =
          u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
      return;
    }
    u32x4 t[3];
    cut3(v, t);
#pragma unroll
    for (int q = 0; q < 3; ++q) *((g_u32x4*)(base + q * plane + off)) = t[q];
  }
};

constexpr int kNoSave = 2;  // a variant's B, beside the kinds: no checkpoint is kept

// a and b of eight columns: s for the down projection, and the checkpoints. Lanes
// past the last column take part in their group with zeros. Variants: the activation,
// and the checkpoints' kind.
struct PrGateOut {
  static constexpr int OPS = 2, AHEAD = 1;
  struct Pre {};
  static MUON_INLINE void settle(const Pre&) {}
  PrLane at;
  Planes s;
  Saved qa, qb, qs;
  int m, n, act;
  MUON_INLINE PrGateOut(PrItemRef it, PrArgsPtr args, PrLane lane)
      : at(lane), s(args->mlp.plane[0], args->mlp, pinned(args->parts), lane), qa(args->mlp.a, lane), qb(args->mlp.b, lane),
        qs(args->mlp.s, lane), m(pinned(it.m)), n(pinned(it.n)), act(pinned(args->mlp.act)) {}
  // All of the checkpoints or none, and s in bf16.
  MUON_INLINE bool plain() const { return s.parts == 1 && !qa.q == !qb.q && !qa.q == !qs.q; }
  template <int ACT, class F>
  MUON_INLINE void dispatch_kind(F f) const {
    if (!qa.q) f(PrVariant<true, ACT, kNoSave>{});
    else if (qa.kind == MUON_Q8_INT8) f(PrVariant<true, ACT, MUON_Q8_INT8>{});
    else f(PrVariant<true, ACT, MUON_Q8_E4M3>{});
  }
  template <class F>
  MUON_INLINE void dispatch(F f) const {
    if (act == MUON_ACT_SILU) dispatch_kind<MUON_ACT_SILU>(f);
    else if (act == MUON_ACT_GELU) dispatch_kind<MUON_ACT_GELU>(f);
    else if (act == MUON_ACT_GELU_TANH) dispatch_kind<MUON_ACT_GELU_TANH>(f);
    else dispatch_kind<MUON_ACT_RELU>(f);
  }
  template <class V>
  MUON_INLINE void pre(int, Pre&) const {}
  template <class V>
  MUON_INLINE void emit(int row, float a[8], float b[8], const Pre&) const {
    const bool there = V::FULL || row + at.row < m;
    const int live = n - at.col;
    float v[8];
    activations<V::A>(a, act, [&](int i, float f, float) __attribute__((always_inline)) { v[i] = f * b[i]; });
    if (!V::FULL && live < 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= live) a[i] = b[i] = v[i] = 0.f;
    }
    if (V::FULL || (there && live > 0)) s.put<V>(row, v);
    if constexpr (!V::FULL || V::B != kNoSave) {
      if (V::FULL || qa.q) qa.save<V>(row, there, a);
      if (V::FULL || qb.q) qb.save<V>(row, there, b);
      if (V::FULL || qs.q) qs.save<V>(row, there, v);
    }
  }
};

// ds of eight columns, with a and b from their checkpoints. Variants as above.
struct PrGateGradOut {
  static constexpr int OPS = 1, AHEAD = 8;
  struct Pre {
    u32x2 a, b;
    uint32_t ea, eb;
  };
  static MUON_INLINE void settle(const Pre& p) { asm volatile("" ::"v"(p.a), "v"(p.b), "v"(p.ea), "v"(p.eb)); }
  PrLane at;
  Saved qa, qb;
  Planes pa, pb;
  char *da, *db;
  int64_t lda, ldb;
  uint32_t offa, offb;
  int m, live, act;
  bool f32;
  MUON_INLINE PrGateGradOut(PrItemRef it, PrArgsPtr args, PrLane lane)
      : at(lane), qa(args->mlp.a, lane), qb(args->mlp.b, lane), pa(args->mlp.plane[0], args->mlp, pinned(args->parts), lane),
        pb(args->mlp.plane[1], args->mlp, pinned(args->parts), lane), da(static_cast<char*>(pinned(args->mlp.d[0]))),
        db(static_cast<char*>(pinned(args->mlp.d[1]))), lda(pinned(args->mlp.ldd[0])), ldb(pinned(args->mlp.ldd[1])),
        m(pinned(it.m)), live(it.n - lane.col), act(pinned(args->mlp.act)), f32(pinned(args->f32)) {
    const int shift = f32 ? 2 : 1;
    offa = ((uint32_t)at.row * (uint32_t)lda + (uint32_t)at.col) << shift;
    offb = ((uint32_t)at.row * (uint32_t)ldb + (uint32_t)at.col) << shift;
    lda <<= shift;
    ldb <<= shift;
  }
  MUON_INLINE bool plain() const { return !f32 && !pa.p; }  // da and db are the next product's operands as they are
  template <int ACT, class F>
  MUON_INLINE void dispatch_kind(F f) const {
    if (qa.kind == MUON_Q8_INT8) f(PrVariant<true, ACT, MUON_Q8_INT8>{});
    else f(PrVariant<true, ACT, MUON_Q8_E4M3>{});
  }
  template <class F>
  MUON_INLINE void dispatch(F f) const {
    if (act == MUON_ACT_SILU) dispatch_kind<MUON_ACT_SILU>(f);
    else if (act == MUON_ACT_GELU) dispatch_kind<MUON_ACT_GELU>(f);
    else if (act == MUON_ACT_GELU_TANH) dispatch_kind<MUON_ACT_GELU_TANH>(f);
    else dispatch_kind<MUON_ACT_RELU>(f);
  }
  template <class V>
  MUON_INLINE void pre(int row, Pre& p) const {
    if (!V::FULL && (row + at.row >= m || live <= 0)) return;
    qa.load(row, p.a, p.ea);
    qb.load(row, p.b, p.eb);
  }
  template <class V>
  MUON_INLINE void emit(int row, float ds[8], float*, const Pre& p) const {
    if (!V::FULL && (row + at.row >= m || live <= 0)) return;
    float a[8], b[8], ga[8], gb[8];
    q8_decode(p.a, p.ea, V::FULL ? V::B : qa.kind, a);
    q8_decode(p.b, p.eb, V::FULL ? V::B : qb.kind, b);
    activations<V::A>(a, act, [&](int i, float f, float df) __attribute__((always_inline)) {
      ga[i] = ds[i] * b[i] * df;
      gb[i] = ds[i] * f;
    });
    char *ba = da + (int64_t)row * lda, *bb = db + (int64_t)row * ldb;
    if constexpr (V::FULL) {
      store_run(reinterpret_cast<u16*>(ba + offa), 8, ga);
      store_run(reinterpret_cast<u16*>(bb + offb), 8, gb);
      return;
    }
    if (f32) {
      store_run(reinterpret_cast<float*>(ba + offa), live, ga);
      store_run(reinterpret_cast<float*>(bb + offb), live, gb);
    } else {
      store_run(reinterpret_cast<u16*>(ba + offa), live, ga);
      store_run(reinterpret_cast<u16*>(bb + offb), live, gb);
    }
    if (pa.p) {
      if (live < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i >= live) ga[i] = gb[i] = 0.f;
      }
      pa.put<V>(row, ga);
      pb.put<V>(row, gb);
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

// A thread takes octets of columns of one operand, all workgroups' worth apart: one
// while there are few, then up to 8. One launch for all operands of a call. Bound by
// memory: 4 and 6 bytes per fp32 element, 12.6 M of them in 22 us (5.7 TB/s).
constexpr int kPackOctets = 8, kPackFew = 1024;  // per thread; workgroups

template <class T, int PARTS>
__global__ void __launch_bounds__(256) pack_kernel(PrPacks args) {
  int i = 0;
  for (int j = 1; j < args.n; ++j) i += (int)blockIdx.x >= args.pack[j].first;
  const PrPack& p = args.pack[i];
  const int64_t count = p.octets * p.rows, blocks = (i + 1 < args.n ? args.pack[i + 1].first : args.blocks) - p.first;
  const T* src = static_cast<const T*>(p.src);
  for (int64_t at = (int64_t)((int)blockIdx.x - p.first) * 256 + threadIdx.x; at < count; at += blocks * 256) {
    const int64_t row = count <= INT32_MAX ? (uint32_t)at / (uint32_t)p.octets : at / p.octets, col = (at - row * p.octets) * 8;
    float v[8];
    load_run(src + row * p.ld + col, p.cols - (int)col, v);
    u16* to = static_cast<u16*>(p.dst) + at * 8;
    if constexpr (PARTS == 1) {
      *((g_u32x4*)to) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    } else {
      u32x4 t[3];
      cut3(v, t);
#pragma unroll
      for (int q = 0; q < 3; ++q) *((g_u32x4*)(to + q * count * 8)) = t[q];
    }
  }
}

hipError_t launch_packs(const PrPacks& args, bool f32, hipStream_t s) {
  if (args.n == 0) return hipSuccess;
  PrPacks a = args;
  a.blocks = 0;
  for (int i = 0; i < a.n; ++i) {
    const int64_t each = (a.pack[i].octets * a.pack[i].rows + 255) / 256, want = (each + kPackOctets - 1) / kPackOctets;
    a.pack[i].first = a.blocks;
    a.blocks += (int)(each < kPackFew ? each : want < kPackFew ? kPackFew : want < 8192 ? want : 8192);
  }
  if (f32) hipLaunchKernelGGL((pack_kernel<float, 3>), dim3(a.blocks), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((pack_kernel<u16, 1>), dim3(a.blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_mlp(const PrArgs& args, int epilogue, bool transposed_b, hipStream_t s) {
  if (epilogue == kPrGate) return launch_tiles<kNT16, PrGateOut>(args, s);
  if (epilogue == kPrGateGrad) return launch_tiles<kNN16, PrGateGradOut>(args, s);
  return transposed_b ? launch_tiles<kNN16, PrStoreOut>(args, s) : launch_tiles<kNT16, PrStoreOut>(args, s);
}

}  // namespace muon
