// The tile engine of the layers' products on gfx950, C[m][n] = sum_k A[m][k] B[n][k]
// (or B[k][n]), and the way its tiles leave: shared by the kernels of the gated
// block and of the 8-bit linear product.
//
// A workgroup of four waves, 2 x 2, sums one BM x BN tile, or a piece of its sum,
// in MFMA accumulators. A stage is RB bytes of K of every row of both operands,
// copied global -> LDS directly, in a ring of ST stages; the copies of later
// stages and the fragments of the next sub-step go between the MFMAs, in a fixed
// order. Then the tile goes through LDS once more in fp32, so that a thread holds
// eight consecutive columns of a row, which is what an epilogue works on: a store
// instruction covers whole lines, and a group of a checkpoint is four lanes.
//
// Bound by the matrix units and what goes between their instructions: 256 x 256 tiles
// with one wave per SIMD, 1200 to 1250 TFLOP/s in bf16 (4096 x 5120 x 25600: 881 us; MFMA
// busy 60% of the cycles at 1.9 GHz, near the power limit) and 2200 in 8 bits (8192 x
// 25600 x 5120: 976 us, 51%). Smaller tiles where there are fewer: 128 x 128, two
// workgroups per CU, and 64 x 64. They are bound by LDS, which a stage's copies and
// fragments keep busy 1.5 and 3 times as long as its MFMAs the matrix units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device.h"
#include "layer_internal.h"
#include "product_internal.h"
#include "q8.h"

namespace muon {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef const __attribute__((address_space(4))) PrArgs* PrArgsPtr;
typedef const __attribute__((address_space(4))) PrItem& PrItemRef;
typedef uint32_t __attribute__((aligned(1))) u32_any;
typedef u32_any __attribute__((address_space(1))) g_u32_any;

// kNT16, kNN16: bf16 operands, B as n x k or as k x n. kNT8: e4m3 operands with
// scales, in the 8-bit MFMA that applies them: twice the rate, but it adds 16 products
// of consecutive k on a common grid of 2^-13 of the largest (measured: with 1 in such a
// run, 2^-13 counts and 2^-14 does not; a relative error of about 5e-5 in a sum).
// kNT8X, for fp32 results: the same operands decoded to bf16, exactly, on their way
// from LDS, and the bf16 MFMA.
enum PrMode { kNT16, kNN16, kNT8, kNT8X };

// The slot of 16-byte chunk c of row r in an LDS row of 8 slots is c ^ swz(r): the
// rows that the lanes of a fragment read together lie in different banks.
MUON_INLINE int pr_swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }
// The same for a row of K of a transposed B, read four rows at a time.
template <int BN>
MUON_INLINE int pr_swz_k(int r) {
  if constexpr (BN >= 128) return lds_swizzle_k(r);
  else return (r & 3) << 1;
}

template <int BM_, int BN_, int RB_, int ST_, int MODE_, int WG_>
struct PrCfg {
  static constexpr int BM = BM_, BN = BN_, RB = RB_, ST = ST_, MODE = MODE_, WG = WG_;  // WG: workgroups per CU
  static constexpr int NT = 256, NW = 4;
  static constexpr int WM = BM / 2, WN = BN / 2, FM = WM / 32, FN = WN / 32;
  static constexpr bool F8 = MODE == kNT8 || MODE == kNT8X, NN = MODE == kNN16;
  static constexpr int BK = RB / (F8 ? 1 : 2);       // elements of K per stage
  static constexpr int S = RB / 16;                  // 16-byte slots of a row
  static constexpr int AB = BM * RB, BB = BN * RB, STAGE = AB + BB, RING = ST * STAGE;
  static constexpr int DA = AB / 1024 / NW, DB = BB / 1024 / NW, PS = DA + DB;  // copies per wave and stage
  static constexpr int RPI = 1024 / RB;              // rows of one copy
  static constexpr int BROW = BN * 2, BRPI = 1024 / BROW, BS = BN / 8;  // the same of a transposed B
  static constexpr int SUB = MODE == kNT8 ? 64 : MODE == kNT8X ? 16 : 32;  // bytes of K of a sub-step
  static constexpr int KK = RB / SUB, PER = FM * FN, SLOTS = KK * PER, NF = FM + FN;
  // Small tiles have too few MFMAs in a sub-step to cover a read from LDS: they hold the
  // fragments of two whole stages (4096 x 2048 x 6144 in 64 x 64 tiles 165 us, with those
  // of two sub-steps 174; few tiles gain 0 to 5%).
  static constexpr bool AHEAD = PER <= 4;
  static constexpr int KF = AHEAD ? KK : 1;
  // The slot at which the workgroup meets: this stage's fragments are in registers, the
  // next stage must be in LDS.
  static constexpr int MEET = AHEAD ? (PER == 1 ? 0 : SLOTS / 2) : SLOTS - 4;
  // 8-bit operands: exponents of 1024 of K, for as many runs of stages as a ring can
  // hold parts of
  static constexpr int CHUNK = 1024 / RB, TABS = ST, EX_A = 8 * BM * 4, EX_B = 8 * 2 * 4, EX = F8 ? TABS * (EX_A + EX_B) : 0;
  static constexpr int LDS = RING + EX;
  // The tile leaves through the stage that it used last (the others hold the next
  // tile's first stages), which is as large as one block of 32 rows of every wave.
  static constexpr int PASSES = FM;
  static_assert(RB == kBlock, "a stage's row is 8 slots, and 128 of K in 8 bits: one scale of a weight's");
  static_assert(BM == BN && 64 * BN * 4 == STAGE, "a pass fills a stage");
  static_assert(KK % 2 == 0 && (AHEAD || MEET >= SLOTS - PER) && (AHEAD || MODE != kNT8X), "schedule assumptions");
  static_assert(DA % 2 == 0 && DB % 2 == 0 && (ST & (ST - 1)) == 0, "copies of A and B lie alike");
  typedef std::conditional_t<MODE == kNT8, i32x8, std::conditional_t<MODE == kNT8X, u32x2, bf16x8>> Frag;  // as read
};

// The item that number `unit` of a numbering over the items belongs to.
template <class P>
MUON_INLINE int pr_item(P first, int unit) {
  int idx = 0;
#pragma unroll
  for (int i = 1; i < kPrItems; ++i) idx += unit >= first[i];
  return __builtin_amdgcn_readfirstlane(idx);
}
// Tile (tm, tn) of local tile number t: bands of 4 tile rows walked column by
// column, so 32 consecutive tiles cover 4 x 8.
MUON_INLINE void pr_tile(int t, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int band = (uint32_t)t / (uint32_t)(4 * tiles_n), r = t - band * 4 * tiles_n;
  const int h = min(4, tiles_m - 4 * band);
  tn = (uint32_t)r / (uint32_t)h;
  tm = 4 * band + (r - tn * h);
}

// Which planes the p-th of the six products of two fp32 numbers takes, smallest
// products first (0 lo, 1 mid, 2 hi): lo hi, hi lo, mid mid, mid hi, hi mid, hi
// hi. What is left out is below 2^-24 of hi hi.
MUON_INLINE int pr_plane_a(int p) { return p == 0 ? 0 : p == 1 ? 2 : p == 2 ? 1 : p == 3 ? 1 : 2; }
MUON_INLINE int pr_plane_b(int p) { return p == 0 ? 2 : p == 1 ? 0 : p == 2 ? 1 : p == 3 ? 2 : p == 4 ? 1 : 2; }

// A unit of a launch: a tile, or a piece of its sum.
struct PrUnit {
  int idx, piece, m0, n0, begin, total;  // item; piece of it (or -1); first row and column; first stage and how many
};
template <class Z>
MUON_INLINE PrUnit pr_unit(PrArgsPtr args, bool whole, int unit) {
  PrUnit u;
  u.idx = whole ? pr_item(args->whole0, unit) : pr_item(args->piece0, unit);
  PrItemRef it = args->item[u.idx];
  int tile;
  if (whole) {
    u.piece = -1;
    tile = unit - args->whole0[u.idx];
    u.begin = 0;
    u.total = it.stages;
  } else {
    // the first of a tile's pieces are one stage longer, where the stages do not divide
    const int rest = it.tiles_m * it.tiles_n - it.whole, more = it.stages - it.per * it.splits;
    u.piece = unit - args->piece0[u.idx];
    const int split = (uint32_t)u.piece / (uint32_t)rest;
    tile = it.whole + u.piece - split * rest;
    u.begin = split * it.per + min(split, more);
    u.total = it.per + (split < more);
  }
  int tm, tn;
  pr_tile(tile, it.tiles_m, it.tiles_n, tm, tn);
  u.m0 = tm * Z::BM;
  u.n0 = tn * Z::BN;
  return u;
}

// Columns of a tile that a thread holds together, and the rest of an epilogue's
// common side.
constexpr int kRun = 8;

template <class T>
MUON_INLINE void load_run(const T* p, int live, float v[8]) {  // p at any alignment of T; past `live` columns 0
  if (live >= 8) {
    if constexpr (sizeof(T) == 4) {
      const u32x4 lo = gload16_any(p), hi = gload16_any(p + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = __uint_as_float(lo[i]);
        v[4 + i] = __uint_as_float(hi[i]);
      }
    } else {
      const u32x4 w = gload16_any(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < live ? Elem<T>::load(p + i) : 0.f;
  }
}
template <class T>
MUON_INLINE void store_run(T* p, int live, const float v[8]) {
  if (live >= 8) {
    if constexpr (sizeof(T) == 4) {
      gstore16_any(p, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
      gstore16_any(p + 4, u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])});
    } else {
      gstore16_any(p, u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])});
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < live) Elem<T>::store(p + i, v[i]);
  }
}

// The same for eight bf16 past the caches, which leaves them to the operands: for
// outputs of more than the 32 MB that all L2s hold. 8-bit products both ways, inputs
// saved before: 8192 x 25600 x 5120 2228 -> 2168 us, 4096 x 6144 x 2048 (one of two outputs)
// 186.8 -> 183.6; with smaller outputs stored so too 1024 x 8192 x 5120 167.4 -> 169.8.
constexpr int64_t kStreamFrom = int64_t(16) << 20;  // elements
MUON_INLINE void stream_run(void* p, const float v[8]) {
  __builtin_nontemporal_store(
      u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])}, (g_u32x4_any*)p);
}

// How an epilogue takes a tile apart. A thread holds eight consecutive columns of one
// row at a time: its row is `row` plus one that all threads share, its first column
// always col. The addresses are then a scalar and a 32-bit offset that does not change.
//
// An epilogue comes in variants: PrAny takes every tile and looks at everything as it
// goes; the others are for tiles without an edge, and know what they look at. They
// have no branch that may leave out a load or a store, so that a wait is for what it
// needs and not for all that may be in flight.
struct PrLane {
  int row, col;
};
template <bool FULL_, int A_ = -1, int B_ = -1>
struct PrVariant {
  static constexpr bool FULL = FULL_;
  static constexpr int A = A_, B = B_;
};
typedef PrVariant<false> PrAny;

// Values that stay in scalar registers: read again from the kernel's arguments, they
// would cost a wait each.
template <class T>
MUON_INLINE T pinned(T v) {
  asm volatile("" : "+s"(v));
  return v;
}

// C's store: eight columns of a row, plus beta times those of c, rounded once.
struct PrStoreOut {
  static constexpr int OPS = 1, AHEAD = 8;
  struct Pre {
    uint32_t c[8];  // of a whole tile as it came (what is done with it would wait for it), else fp32
  };
  PrLane at;
  char* out;
  const char* c;
  int64_t ldo, ldc;
  int m, live;
  float beta;
  bool f32, stream;
  uint32_t off, offc;
  MUON_INLINE PrStoreOut(PrItemRef it, PrArgsPtr a, PrLane lane) : at(lane) {
    out = static_cast<char*>(pinned(it.out));
    c = static_cast<const char*>(pinned(it.c));
    ldo = pinned(it.ldo);
    ldc = pinned(it.ldc);
    m = pinned(it.m);
    beta = pinned(it.beta);
    f32 = pinned(a->f32);
    live = it.n - at.col;
    stream = (int64_t)m * it.n > kStreamFrom;
    const int shift = f32 ? 2 : 1;
    off = ((uint32_t)at.row * (uint32_t)ldo + (uint32_t)at.col) << shift;
    offc = ((uint32_t)at.row * (uint32_t)ldc + (uint32_t)at.col) << shift;
    ldo <<= shift;
    ldc <<= shift;
  }
  MUON_INLINE bool plain() const { return true; }
  // Variants: A the type (1 fp32), B whether there is a c (1) and bf16 streams (2).
  template <class F>
  MUON_INLINE void dispatch(F f) const {
    if (f32) beta != 0.f ? f(PrVariant<true, 1, 1>{}) : f(PrVariant<true, 1, 0>{});
    else if (stream) beta != 0.f ? f(PrVariant<true, 0, 3>{}) : f(PrVariant<true, 0, 2>{});
    else beta != 0.f ? f(PrVariant<true, 0, 1>{}) : f(PrVariant<true, 0, 0>{});
  }
  template <class V>
  MUON_INLINE void pre(int row, Pre& p) const {
    const char* at_c = c + (int64_t)row * ldc + offc;
    if constexpr (V::FULL) {
      // before the variant is known, both halves of what an fp32 c would need, if there is a c
      if (V::B < 0 ? beta != 0.f : V::B & 1) {
        const u32x4 lo = gload16_any(at_c), hi = V::A == 0 || (V::A < 0 && !f32) ? lo : gload16_any(at_c + 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p.c[i] = lo[i];
          p.c[4 + i] = hi[i];
        }
      }
    } else if (beta != 0.f && row + at.row < m && live > 0) {
      float x[8];
      if (f32) load_run(reinterpret_cast<const float*>(at_c), live, x);
      else load_run(reinterpret_cast<const u16*>(at_c), live, x);
#pragma unroll
      for (int i = 0; i < kRun; ++i) p.c[i] = __float_as_uint(x[i]);
    }
  }
  static MUON_INLINE void settle(const Pre& p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) asm volatile("" ::"v"(p.c[i]));
  }
  // c as fp32 (WIDE), or as packed bf16.
  template <bool WIDE>
  MUON_INLINE void add(const Pre& p, float v[8]) const {
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const float x = __uint_as_float(WIDE ? p.c[i] : i & 1 ? p.c[i / 2] & 0xffff0000u : p.c[i / 2] << 16);
      v[i] = fmaf(beta, x, v[i]);
    }
  }
  template <class V>
  MUON_INLINE void emit(int row, float v[8], float*, const Pre& p) const {
    char* to = out + (int64_t)row * ldo + off;
    if constexpr (V::FULL) {
      if constexpr (V::B & 1) add<V::A != 0>(p, v);
      if constexpr (V::A != 0) store_run(reinterpret_cast<float*>(to), 8, v);
      else if constexpr (V::B & 2) stream_run(to, v);
      else store_run(reinterpret_cast<u16*>(to), 8, v);
    } else {
      if (row + at.row >= m || live <= 0) return;
      if (beta != 0.f) add<true>(p, v);
      if (f32) store_run(reinterpret_cast<float*>(to), live, v);
      else store_run(reinterpret_cast<u16*>(to), live, v);
    }
  }
};

// A tile's way out: its partial sums, BM x BN floats, or the epilogue Out. Through
// LDS, a pass of 32 rows of every wave at a time: staged row r is row WM*(r / 32) +
// 32*pass + r % 32 of the tile; its 16-byte unit u sits at u ^ (r % the row's units).
template <class Z>
struct PrStage {
  static constexpr int MASK = Z::BN / 4 - 1, ROWS = 64;
  unsigned char* lds;
  const f32x16 (&acc)[Z::FM][Z::FN];
  // The first of the tile's rows that belong to staged row r (a multiple of what a
  // pass's threads share).
  MUON_INLINE static int tile_row(int pass, int r) { return Z::WM * (r / 32) + 32 * pass + r % 32; }
  // One pass's rows. The marks at both ends keep the passes apart: the compiler would
  // make one of them all, with a pointer to the sums, which then live in memory.
  template <int P>
  MUON_INLINE void fill_from() const {
    asm volatile("; pass %0" ::"n"(P) : "memory");
    const int tid = fresh_tid(), lane = tid & 63, wave = tid >> 6, wm = wave >> 1, wn = wave & 1;
#pragma unroll
    for (int j = 0; j < Z::FN; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int r = wm * 32 + (lane & 31), u = wn * (8 * Z::FN) + 8 * j + 2 * g + (lane >> 5);
        const f32x16& t = acc[P][j];
        *reinterpret_cast<f32x4*>(lds + r * Z::BN * 4 + ((u ^ (r & MASK)) << 4)) =
            f32x4{t[4 * g], t[4 * g + 1], t[4 * g + 2], t[4 * g + 3]};
      }
    asm volatile("; pass %0" ::"n"(P) : "memory");
  }
  template <int P>
  MUON_INLINE void fill_if(int pass) const {
    if constexpr (P < Z::PASSES) {
      if (pass == P) fill_from<P>();
      fill_if<P + 1>(pass);
    }
  }
  // The barrier before is for the readers of the pass before.
  MUON_INLINE void fill(int pass) const {
    if (pass) __syncthreads();
    fill_if<0>(pass);
    __syncthreads();
  }
  MUON_INLINE void run(int r, int col, float v[8]) const {
    const unsigned char* row = lds + r * Z::BN * 4;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const f32x4 t = *reinterpret_cast<const f32x4*>(row + (((col / 4 + q) ^ (r & MASK)) << 4));
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * q + e] = t[e];
    }
  }
};

// Where a tile's two products lie side by side (DUAL), the waves' left column holds
// the first and the right one the second.
template <class Z, class Out, bool FULL>
MUON_INLINE void pr_leave_as(const PrStage<Z>& stage, const Out& out, int m0) {
  constexpr bool DUAL = Out::OPS == 2;
  constexpr int COLS = DUAL ? Z::BN / 2 : Z::BN, LW = COLS / kRun;
  constexpr int STEP = Z::NT / LW, IT = PrStage<Z>::ROWS / STEP, PRE = IT < Out::AHEAD ? IT : Out::AHEAD, ALL = Z::PASSES * IT;
  static_assert(IT >= 1 && IT % PRE == 0 && (32 % STEP == 0 || STEP % 32 == 0), "the threads of a pass take whole rows");
  const int tid = fresh_tid(), row = tid / LW, col = tid % LW * kRun;
  // The matrix's row of run g, without the thread's own part.
  auto row_of = [&](int g) __attribute__((always_inline)) { return m0 + PrStage<Z>::tile_row(g / IT, g % IT * STEP); };
  typename Out::Pre pre[PRE];
#pragma unroll
  for (int g = 0; g < PRE; ++g) out.template pre<PrVariant<FULL>>(row_of(g), pre[g]);
#pragma unroll 1
  for (int pass = 0; pass < Z::PASSES; ++pass) {
    stage.fill(pass);
    auto runs = [&](auto variant) __attribute__((always_inline)) {
      typedef decltype(variant) V;
#pragma unroll 1
      for (int q0 = 0; q0 < IT; q0 += PRE)
#pragma unroll
        for (int a = 0; a < PRE; ++a) {
          const int g = pass * IT + q0 + a, n = min(g + PRE, ALL - 1);  // past the end: the last one again
          float v[8], w[8];
          stage.run((q0 + a) * STEP + row, col, v);
          if constexpr (DUAL) stage.run((q0 + a) * STEP + row, COLS + col, w);
          out.template emit<V>(row_of(g), v, w, pre[a]);
          out.template pre<V>(row_of(n), pre[a]);
          __builtin_amdgcn_sched_barrier(0);
        }
    };
    if constexpr (FULL) out.dispatch(runs);
    else runs(PrAny{});
  }
  // The loads past the end come in here: in flight, they would be waited for where
  // their registers are next written, in the next tile's stages.
#pragma unroll
  for (int g = 0; g < PRE; ++g) Out::settle(pre[g]);
}

template <class Z, class Out>
MUON_INLINE void pr_leave(PrArgsPtr args, PrItemRef it, int piece, int m0, int n0, unsigned char* lds,
                          const f32x16 (&acc)[Z::FM][Z::FN]) {
  constexpr bool DUAL = Out::OPS == 2;
  constexpr int COLS = DUAL ? Z::BN / 2 : Z::BN, LW = COLS / kRun;
  const int tid = fresh_tid(), c0 = DUAL ? n0 >> 1 : n0;
  const PrStage<Z> stage{lds, acc};
  if (piece >= 0) {
    constexpr int PLW = Z::BN / kRun, PSTEP = Z::NT / PLW;
    const int row = tid / PLW, col = tid % PLW * kRun;
    float* part = args->partial + (int64_t)(it.part0 + piece) * Z::BM * Z::BN + PrStage<Z>::tile_row(0, row) * Z::BN + col;
#pragma unroll 1
    for (int pass = 0; pass < Z::PASSES; ++pass) {
      stage.fill(pass);
#pragma unroll 4
      for (int q = 0; q < PrStage<Z>::ROWS / PSTEP; ++q) {
        float v[8];
        stage.run(q * PSTEP + row, col, v);
        store_run(part + PrStage<Z>::tile_row(pass, q * PSTEP) * Z::BN, 8, v);
      }
    }
    return;
  }
  const Out out(it, args, PrLane{PrStage<Z>::tile_row(0, tid / LW), c0 + tid % LW * kRun});
  if (out.plain() && m0 + Z::BM <= it.m && c0 + (DUAL ? Z::BN / 2 : Z::BN) <= it.n) pr_leave_as<Z, Out, true>(stage, out, m0);
  else pr_leave_as<Z, Out, false>(stage, out, m0);
}

// The arguments lie in host memory, and every line of them is a trip there that the
// tile's prologue and epilogue would take one after the other: all lines that a launch
// of one product reads are asked for at once (a 64 x 64 tile's prologue 5000 -> 4200
// cycles, its epilogue's first step 2200 -> 1450).
MUON_INLINE void pr_touch(PrArgsPtr args) {
  typedef const __attribute__((address_space(4))) uint32_t* Words;
  constexpr int LINE = 16, HEAD = (offsetof(PrArgs, item) + sizeof(PrItem)) / 4, TAIL = offsetof(PrArgs, mlp) / 4, END = sizeof(PrArgs) / 4;
  uint32_t all = 0;
#pragma unroll
  for (int w = 0; w < HEAD; w += LINE) all ^= ((Words)args)[w];
#pragma unroll
  for (int w = TAIL / LINE * LINE; w < END; w += LINE) all ^= ((Words)args)[w];
  asm volatile("" ::"s"(all));
}

// All units of one workgroup. XCD b % 8 gets a contiguous range of the whole tiles and
// one of the pieces, which its workgroups take in turn, so that the tiles that run
// there together share operand panels in its L2. The copies run ST - 1 stages ahead of the sum, across tiles: a
// tile starts with its first stages in LDS, and its predecessor leaves under their
// copies.
template <class Z, class Out>
MUON_INLINE void pr_run(unsigned char* smem) {
  constexpr bool DUAL = Out::OPS == 2;
  constexpr int FM = Z::FM, FN = Z::FN, RB = Z::RB, S = Z::S;
  const PrArgsPtr args = (PrArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
  pr_touch(args);
  const int xcd = blockIdx.x & 7, wholes = args->wholes, pieces = args->pieces;
  const int first_w = xcd * (wholes >> 3) + min(xcd, wholes & 7), count_w = (wholes >> 3) + (xcd < (wholes & 7));
  // the pieces' remainder goes to the XCDs that the wholes' did not reach
  const int turn = (xcd - (wholes & 7)) & 7;
  const int first_p = turn * (pieces >> 3) + min(turn, pieces & 7), count = count_w + (pieces >> 3) + (turn < (pieces & 7));
  auto unit_at = [&](int i) __attribute__((always_inline)) {
    return pr_unit<Z>(args, i < count_w, i < count_w ? first_w + i : first_p + i - count_w);
  };
  const int step = ((int)gridDim.x >> 3) + (xcd < ((int)gridDim.x & 7));
  int at = blockIdx.x >> 3;
  if (at >= count) return;

  const int tid = fresh_tid(), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)smem);
  const int pairs = args->parts == 3 ? 6 : 1;

  // ---- what is copied next: a stage of a unit, at K step `ks` of pair of planes `seg`
  const uint8_t *la = nullptr, *lb0 = nullptr, *lb1 = nullptr;
  int64_t lda = 0, ldb = 0;
  int lat = at - step, lidx = 0, lm0 = 0, ln0 = 0, lks = 0, lseg = 0, lleft = 0, lk = 0, lkt = 1;
  uint32_t limit = 0, limit_k = 0;  // where a row (of a transposed B: the rows) of the stage end
  bool lfresh = false;              // the stage's exponents are not in a table yet
  int ltab = -1;
  // Copy q of an operand fills 1 KB: rows RPI*q .. +RPI-1, lane l slot l % S of row
  // l / S, which holds chunk slot ^ swz(row). Rows past the last one read the last
  // one, and are never stored. In a short stage, chunks past the end of a row read
  // its last chunk (for a transposed B: rows of K past the last one the last one);
  // what is not the product's becomes zero once it is in LDS.
  uint32_t row_a[Z::DA], row_b[Z::DB], ch_a[2], ch_b[2];
  auto limits = [&]() __attribute__((always_inline)) {
    const int kbytes = Z::F8 ? lk : 2 * lk;
    limit = (uint32_t)min((kbytes - lks * RB + 15) / 16, S) * 16 - 16;
    if constexpr (Z::NN) limit_k = (uint32_t)(min(lk - lks * Z::BK, Z::BK) - 1) * (uint32_t)ldb;
    lfresh = Z::F8 && (lfresh || (lks & (Z::CHUNK - 1)) == 0);
    if (Z::F8 && lfresh) ltab = __builtin_amdgcn_readfirstlane((ltab + 1) & (Z::TABS - 1));
  };
  auto seat = [&]() __attribute__((always_inline)) {
    PrItemRef it = args->item[lidx];
    const int sum = lseg / pairs, p = lseg - sum * pairs;
    const int64_t pa = pairs == 6 ? pr_plane_a(p) * it.pa : 0, pb = pairs == 6 ? pr_plane_b(p) * it.pb : 0;
    la = it.a[sum] + pa + (int64_t)lm0 * lda + (int64_t)lks * RB;
    if constexpr (DUAL) {
      lb0 = it.b[0] + pb + (int64_t)(ln0 >> 1) * ldb + (int64_t)lks * RB;
      lb1 = it.b[1] + pb + (int64_t)(ln0 >> 1) * ldb + (int64_t)lks * RB;
    } else if constexpr (Z::NN) {
      lb0 = it.b[sum] + pb + 2 * ln0 + (int64_t)lks * Z::BK * ldb;
    } else {
      lb0 = it.b[sum] + pb + (int64_t)ln0 * ldb + (int64_t)lks * RB;
    }
  };
  auto open = [&]() __attribute__((always_inline)) {  // the next unit's first stage
    lat += step;
    const PrUnit u = unit_at(lat);
    PrItemRef it = args->item[u.idx];
    lidx = u.idx;
    lm0 = u.m0;
    ln0 = u.n0;
    lk = it.k;
    lda = it.lda;
    ldb = it.ldb;
    lkt = (lk + Z::BK - 1) / Z::BK;
    lseg = (uint32_t)u.begin / (uint32_t)lkt;
    lks = u.begin - lseg * lkt;
    lleft = u.total;
    const int rows_a = it.m - lm0, cols_b = DUAL ? it.n - (ln0 >> 1) : it.n - ln0;
#pragma unroll
    for (int p = 0; p < Z::DA; ++p) {
      const int r = (wave * Z::DA + p) * Z::RPI + lane / S;
      row_a[p] = (uint32_t)min(r, rows_a - 1) * (uint32_t)lda;
      if (p < 2) ch_a[p] = ((lane % S) ^ pr_swz(r)) << 4;
    }
#pragma unroll
    for (int p = 0; p < Z::DB; ++p) {
      if constexpr (Z::NN) {
        const int r = (wave * Z::DB + p) * Z::BRPI + lane / Z::BS;
        row_b[p] = (uint32_t)r * (uint32_t)ldb;
        if (p < 2) ch_b[p] = min((lane % Z::BS) ^ pr_swz_k<Z::BN>(r), (cols_b + 7) / 8 - 1) << 4;
      } else {
        const int r = (wave * Z::DB + p) * Z::RPI + lane / S, c = DUAL ? r & (Z::BN / 2 - 1) : r;
        row_b[p] = (uint32_t)min(c, cols_b - 1) * (uint32_t)ldb;
        if (p < 2) ch_b[p] = ch_a[p];
      }
    }
    seat();
    lfresh = true;
    limits();
  };
  // The stage after this one. Past the last unit's last stage that one is copied
  // again, and nothing of it is used.
  auto advance = [&]() __attribute__((always_inline)) {
    lfresh = false;
    if (--lleft == 0) {
      if (lat + step < count) open();
      else lleft = 1;
      return;
    }
    if (++lks == lkt) {
      lks = 0;
      ++lseg;
      seat();
    } else {
      la += RB;
      lb0 += Z::NN ? (int64_t)Z::BK * ldb : (int64_t)RB;
      if constexpr (DUAL) lb1 += RB;
    }
    limits();
  };
  auto copy = [&](uint32_t buf, int d) __attribute__((always_inline)) {
    const bool is_a = d < Z::DA;
    const int p = is_a ? d : d - Z::DA, q = wave * (is_a ? Z::DA : Z::DB) + p;
    const uint8_t* base = is_a ? la : DUAL && q * Z::RPI >= Z::BN / 2 ? lb1 : lb0;
    const uint32_t v = is_a ? row_a[p] + min(ch_a[p & 1], limit)
                       : Z::NN ? min(row_b[p], limit_k) + ch_b[p & 1] : row_b[p] + min(ch_b[p & 1], limit);
    dma16s(base, v, lds0 + buf + (is_a ? 0 : Z::AB) + q * 1024);
  };
  // Exponents (8-bit operands): eight stages of both, one dword of four groups per
  // row of A and stage, one byte per 128 columns of B and stage. Thread t carries row
  // t's; groups past the end of K get 127, whatever they scale is 0.
  uint32_t ev[8], evb = 0;
  auto load_ex = [&]() __attribute__((always_inline)) {
    if constexpr (Z::F8) {
      PrItemRef it = args->item[lidx];
      const int chunk = lks / Z::CHUNK, groups = (lk + kGroup - 1) / kGroup, kblocks = (lk + kBlock - 1) / kBlock;
      if (tid < Z::BM) {
        const uint8_t* row = it.ea + (int64_t)min(lm0 + tid, it.m - 1) * it.lde + 32 * chunk;
        if (32 * chunk + 32 <= groups) {
#pragma unroll
          for (int w = 0; w < 8; ++w) ev[w] = *((const g_u32_any*)(row + 4 * w));
        } else {
#pragma unroll
          for (int w = 0; w < 8; ++w) {
            ev[w] = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const int g = 4 * w + b;
              ev[w] |= (32 * chunk + g < groups ? (uint32_t)*((const g_u8*)(row + g)) : 127u) << (8 * b);
            }
          }
        }
      }
      if (tid < 16) {
        const int nb = ln0 / kBlock + (tid >> 3), kb = 8 * chunk + (tid & 7);
        evb = nb * kBlock < it.n && kb < kblocks ? (uint32_t)*((const g_u8*)(it.eb + nb * it.ldeb_n + kb * it.ldeb_k)) : 127u;
      }
    }
  };
  auto write_ex = [&](int table) __attribute__((always_inline)) {
    if constexpr (Z::F8) {
      unsigned char* t = smem + Z::RING + table * (Z::EX_A + Z::EX_B);
      if (tid < Z::BM)
#pragma unroll
        for (int w = 0; w < 8; ++w) *reinterpret_cast<uint32_t*>(t + (w * Z::BM + tid) * 4) = ev[w];
      if (tid < 16) *reinterpret_cast<uint32_t*>(t + Z::EX_A + tid * 4) = evb;
    }
  };

  // ---- the sum
  f32x16 acc[FM][FN];
  int k = 0, kt = 1, ks = 0, tab = -1;               // of the unit at hand, and its stage
  auto short_stage = [&](int ks_) __attribute__((always_inline)) {
    const int kbytes = Z::F8 ? k : 2 * k;
    return ks_ * RB + RB > kbytes;
  };
  // Zeros behind the end of K, in both operands (the other one may hold an
  // infinity).
  auto clear = [&](int ks_, uint32_t buf) __attribute__((always_inline)) {
    const int left = (Z::F8 ? k : 2 * k) - ks_ * RB; // bytes of K that are there
    constexpr int ROWS = Z::NN ? Z::BM : Z::BM + Z::BN;
    for (int i = tid; i < ROWS * S; i += Z::NT) {
      const int r = i / S, ch = i % S;
      const int br = r < Z::BM ? r : r - Z::BM;
      u32x4* p = reinterpret_cast<u32x4*>(smem + buf + (r < Z::BM ? 0 : Z::AB) + br * RB + ((ch ^ pr_swz(br)) << 4));
      const int have = left - 16 * ch;
      if (have <= 0) {
        *p = u32x4{0u, 0u, 0u, 0u};
      } else if (have < 16) {
        u32x4 v = *p;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int b = have - 4 * w;
          v[w] &= b >= 4 ? ~0u : b <= 0 ? 0u : (1u << (8 * b)) - 1u;
        }
        *p = v;
      }
    }
    if constexpr (Z::NN) {
      const int have = k - ks_ * Z::BK;
      for (int i = tid; i < Z::BK * Z::BS; i += Z::NT)
        if (i / Z::BS >= have) *reinterpret_cast<u32x4*>(smem + buf + Z::AB + i * 16) = u32x4{0u, 0u, 0u, 0u};
    }
    __syncthreads();
  };

  // Fragments. Lane l of a 32-row block reads row l % 32; of a sub-step of 16 bf16
  // its half l / 32 takes chunk 2 kk + half (8 consecutive k), of 64 e4m3 chunks
  // 4 kk + half and 4 kk + 2 + half: the 8-bit MFMA's halves hold k 0-15, 32-47 and
  // 16-31, 48-63, and its scale of half h is that of k 32 h .. 32 h + 31.
  const int r32 = lane & 31, h = lane >> 5, sw = pr_swz(r32);
  const int G = lane >> 4, i16 = lane & 15;
  typename Z::Frag fa[2][Z::KF][FM], fb[2][Z::KF][FN];
  bf16x8 da[2][FM], db[2][FN];                       // kNT8X: a sub-step's, decoded
  uint32_t sa[FM], sb = 127, na[FM], nb_ = 127;      // this stage's scales, and the next one's
  // Fragment f of sub-step kk into buffer b.
  auto read_frag = [&](int b, uint32_t buf, int kk, int f) __attribute__((always_inline)) {
    const bool is_a = f < FM;
    const int i = is_a ? f : f - FM, to = Z::AHEAD ? kk : 0;
    typename Z::Frag v;
    if (Z::NN && !is_a) {
      if constexpr (Z::NN) {
        const int col = wn * Z::WN + 32 * i + 16 * (G & 1) + 4 * (i16 & 3);
        const unsigned char* p = smem + buf + Z::AB + (kk * 16 + 8 * (G >> 1) + (i16 >> 2)) * Z::BROW +
                                 (((col >> 3) ^ pr_swz_k<Z::BN>(i16 >> 2)) << 4) + 8 * (i16 & 1);
        const v4i16 lo = lds_read_tr(p), hi = lds_read_tr(p + 4 * Z::BROW);
        v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      }
    } else {
      const unsigned char* row = smem + buf + (is_a ? (wm * Z::WM + 32 * i + r32) * RB : Z::AB + (wn * Z::WN + 32 * i + r32) * RB);
      if constexpr (Z::MODE == kNT8) {
        const u32x4 lo = *reinterpret_cast<const u32x4*>(row + (((4 * kk + h) ^ sw) << 4));
        const u32x4 hi = *reinterpret_cast<const u32x4*>(row + (((4 * kk + 2 + h) ^ sw) << 4));
        v = i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
      } else if constexpr (Z::MODE == kNT8X) {
        v = *reinterpret_cast<const u32x2*>(row + ((kk ^ sw) << 4) + 8 * h);
      } else {
        v = *reinterpret_cast<const bf16x8*>(row + (((2 * kk + h) ^ sw) << 4));
      }
    }
    if (is_a) fa[b][to][i] = v;
    else fb[b][to][i] = v;
  };
  // kNT8X: fragment f of sub-step kk in buffer b, decoded with the scales xa and xb of
  // its stage.
  auto decode = [&](int b, int kk, int f, const uint32_t (&xa)[FM], uint32_t xb) __attribute__((always_inline)) {
    if constexpr (Z::MODE == kNT8X) {
      const bool is_a = f < FM;
      const int i = is_a ? f : f - FM;
      const Q8Group<MUON_Q8_E4M3> grp(is_a ? (xa[i] >> (8 * (kk >> 1))) & 255u : xb, true);
      const u32x2 w = is_a ? fa[b][kk][i] : fb[b][kk][i], x = grp.bf16x4(w[0]), y = grp.bf16x4(w[1]);
      const bf16x8 v = __builtin_bit_cast(bf16x8, (u32x4{x[0], x[1], y[0], y[1]}));
      if (is_a) da[kk & 1][i] = v;
      else db[kk & 1][i] = v;
    }
  };
  auto read_ex = [&](int ks_, int t_) __attribute__((always_inline)) {
    if constexpr (Z::F8) {
      const unsigned char* t = smem + Z::RING + t_ * (Z::EX_A + Z::EX_B);
      const int row = ks_ & 7;
#pragma unroll
      for (int i = 0; i < FM; ++i)
        na[i] = *reinterpret_cast<const uint32_t*>(t + (row * Z::BM + wm * Z::WM + 32 * i + r32) * 4);
      nb_ = *reinterpret_cast<const uint32_t*>(t + Z::EX_A + (row + 8 * ((wn * Z::WN) / kBlock)) * 4);
    }
  };
  auto take_ex = [&]() __attribute__((always_inline)) {
    if constexpr (Z::F8) {
#pragma unroll
      for (int i = 0; i < FM; ++i) sa[i] = Z::MODE == kNT8 ? na[i] >> 8 * h : na[i];  // groups of 32, 8 bits each
      sb = nb_;
    }
  };
  auto mfma = [&](int b, int kk, int q) __attribute__((always_inline)) {
    const int i = q / FN, j = q % FN, at_k = Z::AHEAD ? kk : 0;
    if constexpr (Z::MODE == kNT8) {
      if (kk == 0)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[b][at_k][j], fa[b][at_k][i], acc[i][j], 0, 0, 0, (int)sb, 0, (int)sa[i]);
      else
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[b][at_k][j], fa[b][at_k][i], acc[i][j], 0, 0, 0, (int)sb, 2, (int)sa[i]);
    } else if constexpr (Z::MODE == kNT8X) {
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(db[kk & 1][j], da[kk & 1][i], acc[i][j], 0, 0, 0);
    } else {
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[b][at_k][j], fa[b][at_k][i], acc[i][j], 0, 0, 0);
    }
  };

  // Holds the MFMAs above this place: to the compiler they are sums that only later
  // code reads, and it moves them there, behind the barrier.
  auto anchor = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        if constexpr (FM * FN >= 16) asm volatile("" : "+a"(acc[i][j]));
        else asm volatile("" : "+v"(acc[i][j]));
      }
  };

  open();
#pragma unroll 1
  for (int s = 0; s < Z::ST - 1; ++s) {
    if (lfresh) {
      load_ex();
      write_ex(ltab);
    }
#pragma unroll
    for (int d = 0; d < Z::PS; ++d) copy(s * Z::STAGE, d);
    advance();
  }
  wait_vmcnt<(Z::ST - 2) * Z::PS>();
  uint32_t cur = 0, to = (Z::ST - 1) * Z::STAGE;     // the ring's stage at hand, and the one that is loaded
  int due = -1, due_tab = 0;                         // stages until the exponents on their way go to that table

#pragma unroll 1
  for (; at < count; at += step) {
    const PrUnit u = unit_at(at);
    PrItemRef it = args->item[u.idx];
    k = it.k;
    kt = (k + Z::BK - 1) / Z::BK;
    ks = (uint32_t)u.begin % (uint32_t)kt;
    tab = (tab + 1) & (Z::TABS - 1);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    __syncthreads();                                 // its first stage is in LDS, and the last tile has left
    if (short_stage(ks)) clear(ks, cur);
    read_ex(ks, tab);
    take_ex();
    // The first stage's fragments, into buffer b.
    auto begin = [&](auto b_) __attribute__((always_inline)) {
      constexpr int b = decltype(b_)::value;
#pragma unroll
      for (int kk = 0; kk < Z::KF; ++kk)
#pragma unroll
        for (int f = 0; f < Z::NF; ++f) read_frag(b, cur, kk, f);
#pragma unroll
      for (int f = 0; f < Z::NF; ++f) decode(b, 0, f, sa, sb);
    };

    // One stage: MFMAs, and between two of them a little of everything else, in a
    // fixed order. What the MFMAs need next is in registers a few MFMAs before: at MEET
    // the workgroup meets, and the next stage's first fragments (AHEAD: all of them) are
    // read under the remaining MFMAs (after the last stage: for nothing). AHEAD: this
    // stage's fragments are in buffer PAR.
    int t = u.total;
    auto stage = [&](auto PAR_) __attribute__((always_inline)) {
      constexpr int PAR = decltype(PAR_)::value;
      const uint32_t after = cur + Z::STAGE == Z::RING ? 0 : cur + Z::STAGE;
      const int ks1 = ks + 1 == kt ? 0 : ks + 1;
      if (lfresh) {
        // a table is due ST - 2 stages later
        if (due >= 0) write_ex(due_tab);
        load_ex();
        due = Z::ST - 2;
        due_tab = ltab;
      }
      if constexpr (Z::MEET == 0) {
#pragma unroll
        for (int d = 0; d < Z::PS; ++d) copy(to, d);
      }
#pragma unroll
      for (int kk = 0; kk < Z::KK; ++kk)
#pragma unroll
        for (int q = 0; q < Z::PER; ++q) {
          const int slot = kk * Z::PER + q, b = Z::AHEAD ? PAR : kk & 1;
          if (slot == Z::MEET) {
            anchor();
            if (Z::F8 && due >= 0) {
              if (due == 0) write_ex(due_tab);
              --due;
            }
            // the next stage's copies are the oldest in flight
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((Z::ST - 2) * Z::PS) : "memory");
            if (t > 1) {
              if (short_stage(ks1)) clear(ks1, after);
              if (Z::F8 && (ks1 & (Z::CHUNK - 1)) == 0) tab = __builtin_amdgcn_readfirstlane((tab + 1) & (Z::TABS - 1));
            }
            read_ex(ks1, tab);
          }
          mfma(b, kk, q);
          if constexpr (Z::AHEAD) {
            constexpr int ALL = Z::KK * Z::NF;
            if (slot >= Z::MEET) {
#pragma unroll
              for (int f = 0; f < ALL; ++f)
                if (f * (Z::SLOTS - Z::MEET) / ALL == slot - Z::MEET) read_frag(PAR ^ 1, after, f / Z::NF, f % Z::NF);
            }
            if constexpr (Z::MODE == kNT8X) {
#pragma unroll
              for (int f = 0; f < Z::NF; ++f)
                if (kk + 1 < Z::KK && f * Z::PER / Z::NF == q) decode(PAR, kk + 1, f, sa, sb);
            }
          } else {
            if (kk + 1 < Z::KK) {
#pragma unroll
              for (int f = 0; f < Z::NF; ++f)
                if (f * Z::PER / Z::NF == q) read_frag(b ^ 1, cur, kk + 1, f);
            }
            if (slot >= Z::MEET) {
#pragma unroll
              for (int f = 0; f < Z::NF; ++f)
                if (f * (Z::SLOTS - Z::MEET) / Z::NF == slot - Z::MEET) read_frag(0, after, 0, f);
            }
          }
          if constexpr (Z::MEET != 0) {
#pragma unroll
            for (int d = 0; d < Z::PS; ++d)
              if (d * Z::MEET / (Z::PS * (Z::ST == 2 && !Z::AHEAD ? 2 : 1)) == slot) copy(to, d);
          }
          if (slot == Z::SLOTS - 1) {
            anchor();
            take_ex();
#pragma unroll
            for (int f = 0; f < Z::NF; ++f) decode(PAR ^ 1, 0, f, sa, sb);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      advance();
      ks = ks1;
      cur = after;
      to = to + Z::STAGE == Z::RING ? 0 : to + Z::STAGE;
      --t;
    };
    typedef std::integral_constant<int, 0> Even;
    typedef std::integral_constant<int, 1> Odd;
    if constexpr (Z::AHEAD) {
      if (t & 1) {
        begin(Odd{});
        stage(Odd{});
      } else {
        begin(Even{});
      }
#pragma unroll 1
      while (t) {
        stage(Even{});
        stage(Odd{});
      }
    } else {
      begin(Even{});
#pragma unroll 1
      while (t) stage(Even{});
    }
    pr_leave<Z, Out>(args, it, u.piece, u.m0, u.n0, smem + to, acc);
  }
  wait_vmcnt<0>();  // the copies past the last stage
}

// Adds the pieces of a tile in order, then the epilogue. A workgroup takes 256 runs of
// eight columns of one tile.
template <class Out>
MUON_INLINE void pr_join_of(int edge) {
  constexpr bool DUAL = Out::OPS == 2;
  const PrArgsPtr args = (PrArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
  const int cols = DUAL ? edge / 2 : edge, lw = cols / kRun, per = edge * lw / 256;  // workgroups per tile
  int b = blockIdx.x, idx = 0;
  for (; idx < args->n_items; ++idx) {
    const int mine = (args->item[idx].tiles_m * args->item[idx].tiles_n - args->item[idx].whole) * per;
    if (b < mine) break;
    b -= mine;
  }
  PrItemRef it = args->item[idx];
  const int tiles = it.tiles_m * it.tiles_n - it.whole, tile = b / per;
  int tm, tn;
  pr_tile(it.whole + tile, it.tiles_m, it.tiles_n, tm, tn);
  const int row0 = (b - tile * per) * (256 / lw), r = threadIdx.x / lw, col = threadIdx.x % lw * kRun;
  const Out out(it, args, PrLane{r, (DUAL ? tn * edge / 2 : tn * edge) + col});
  typename Out::Pre pre;
  out.template pre<PrAny>(tm * edge + row0, pre);
  const float* p = args->partial + ((int64_t)(it.part0 + tile) * edge + row0 + r) * edge + col;
  const int64_t step = (int64_t)tiles * edge * edge;
  float v[8], w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = w[e] = 0.f;
#pragma unroll 4
  for (int s = 0; s < it.splits; ++s) {
    float x[8], y[8];
    load_run(p + s * step, 8, x);
    if constexpr (DUAL) load_run(p + s * step + edge / 2, 8, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] += x[e];
      if constexpr (DUAL) w[e] += y[e];
    }
  }
  out.template emit<PrAny>(tm * edge + row0, v, w, pre);
}

// Workgroups of a launch: as many as the CUs hold at once.
template <class Z>
inline uint32_t pr_grid(const PrArgs& a) {
  return (uint32_t)(a.wholes + a.pieces < 256 * Z::WG ? a.wholes + a.pieces : 256 * Z::WG);
}
// Workgroups of a launch's join.
inline int64_t pr_join_blocks(const PrArgs& a, bool dual) {
  const int edge = kPrEdge[a.tile];
  int64_t n = 0;
  for (int i = 0; i < a.n_items; ++i)
    n += (int64_t)(a.item[i].tiles_m * a.item[i].tiles_n - a.item[i].whole) * (edge * (dual ? edge / 2 : edge) / kRun / 256);
  return n;
}

}  // namespace muon
