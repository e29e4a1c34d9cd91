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

// Geometry of a tile of EDGE x EDGE outputs: stages of 64 tokens, EDGE bf16
// columns per operand. dY has a ring of three buffers, since its copies run two
// stages ahead; X, which waits in registers, has two. 256: all of a CU's 160 KB
// and eight waves, 2 rows of 4, each of 128 x 64 outputs. 128: half of that,
// two workgroups of four waves per CU, each wave 64 x 64.
template <int EDGE>
struct Geo {
  static constexpr int NW = EDGE / 32, NT = 64 * NW;
  static constexpr int ROW = EDGE * 2;               // bytes of an LDS row
  static constexpr int OP = kWgStep * ROW;           // one operand of a stage
  static constexpr int DY_BUFS = 3, X_BUFS = 2;
  static constexpr int LDS = (DY_BUFS + X_BUFS) * OP;
  static constexpr int FM = EDGE / 64, NB = 2;       // 32-row blocks of dY and of X per wave
  static constexpr int DMA = OP / 1024 / NW;         // copies of dY per wave and stage
  static constexpr int DMA_ROWS = 1024 / ROW;        // token rows of one copy
  static constexpr int ROW_CHUNKS = EDGE / 16;       // 16-byte checkpoint chunks of a token row
  static constexpr int ROW_STEP = NT / ROW_CHUNKS;   // token rows between a thread's chunks
  static constexpr int CHUNKS = kWgStep / ROW_STEP;  // chunks per thread
  static constexpr int PER = FM * NB, SLOTS = 4 * PER, MEET = SLOTS - FM - NB;
  static constexpr int DEC0 = EDGE == 256 ? 3 : 2, DEC = EDGE == 256 ? 3 : 1;  // decoding: first slot, spacing
};

typedef const __attribute__((address_space(4))) WgArgs* ArgsPtr;

// The unit of workgroup b: XCD b % 8 gets a contiguous range of units, so that
// the tiles that run there together share operand panels in its L2.
MUON_INLINE int xcd_unit(int b, int units) {
  const int x = b & 7, i = b >> 3, per = units >> 3, rest = units & 7;
  return x * per + min(x, rest) + i;
}

// The item of a unit, from one scalar load of all first units.
MUON_INLINE int item_of(ArgsPtr a, int unit) {
  int idx = 0;
#pragma unroll
  for (int i = 1; i < kWgItems; ++i) idx += unit >= a->unit0[i];
  return idx;
}

// Tile (tn, tk) of local tile number t: bands of 4 tile rows walked column by
// column, so 32 consecutive tiles cover 4 x 8.
MUON_INLINE void tile_of(int t, int tiles_n, int tiles_k, int& tn, int& tk) {
  const int band = t / (4 * tiles_k), r = t - band * 4 * tiles_k;
  const int h = min(4, tiles_n - 4 * band);
  tk = r / h;
  tn = 4 * band + (r - tk * h);
}

// The gradient's side of a kernel. A row of a tile is stored by LW lanes of
// four columns each: consecutive ones, as one vector, where a row of the
// gradient is a multiple of four long, and otherwise every LW-th, so that a
// store instruction still covers whole lines.
// NT: nontemporal stores, for tiles that all CUs store at once: on one GPU the
// seven 1.7B-layer gradients over 4096 tokens took 362 us with them, 372 without.
template <int LW, bool NT = false>
struct GradOut {
  const __attribute__((address_space(4))) WgItem& it;
  bool g_f32, vec;
  int lane, k0;
  float scale[4];

  MUON_INLINE GradOut(const __attribute__((address_space(4))) WgItem& item, ArgsPtr a, int lane_, int k0_)
      : it(item), g_f32(a->g_f32), vec((item.k & 3) == 0), lane(lane_), k0(k0_) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      scale[i] = 1.f;
      if (it.scale && k0 + col(i) < it.k)
        scale[i] = a->dy_f32 ? Elem<float>::load(static_cast<const float*>(it.scale) + k0 + col(i))
                             : Elem<u16>::load(static_cast<const u16*>(it.scale) + k0 + col(i));
    }
  }
  // Column i of this lane, within the tile.
  MUON_INLINE int col(int i) const { return vec ? 4 * lane + i : lane + LW * i; }
  // This lane's columns (or, with four, 4*lane .. 4*lane+3 anyway) of a row in
  // LDS whose 16-byte unit u, columns 4u .. 4u+3, is at unit(u).
  template <class F>
  MUON_INLINE void gather(float v[4], F unit, bool four) const {
    if (vec || four) {
      const f32x4 t = *reinterpret_cast<const f32x4*>(unit(lane));
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = t[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = unit(col(i) >> 2)[col(i) & 3];
    }
  }
  // Row n of the gradient: the sums v of this lane's columns.
  MUON_INLINE void store(int n, const float v[4]) const {
    if (n >= it.n || k0 + col(0) >= it.k) return;
    const int64_t at = (int64_t)n * it.k + k0;
    float o[4], c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = v[i] * scale[i];
    if (it.beta != 0.f) {
      if (g_f32) load(static_cast<const float*>(it.c) + at, c);
      else load(static_cast<const u16*>(it.c) + at, c);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] += it.beta * c[i];
    }
    if (g_f32) put(static_cast<float*>(it.g) + at, o);
    else put(static_cast<u16*>(it.g) + at, o);
  }
  template <class T>
  MUON_INLINE void load(const T* p, float c[4]) const {
    if (vec) {
      Vec4<T>::load(p + 4 * lane, c);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (k0 + col(i) < it.k) c[i] = Elem<T>::load(p + col(i));
    }
  }
  template <class T>
  MUON_INLINE void put(T* p, const float o[4]) const {
    if (vec && NT) {
      if constexpr (sizeof(T) == 4)
        __builtin_nontemporal_store(f32x4{o[0], o[1], o[2], o[3]}, (g_f32x4*)(p + 4 * lane));
      else
        __builtin_nontemporal_store(u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])}, (g_u32x2*)(p + 4 * lane));
    } else if (vec) {
      Vec4<T>::store(p + 4 * lane, o);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (k0 + col(i) < it.k) Elem<T>::store(p + col(i), o[i]);
    }
  }
};

// One 256 x 256 tile, or one piece of its sum, per workgroup: the largest tile
// whose sums fit a CU's registers, so that a byte of dY or X moved to LDS feeds
// the most MFMAs. Eight waves, two per SIMD, because decoding, fragment reads,
// copies and address arithmetic take nearly as many issue slots as one wave has
// beside its MFMAs: 1902 us against 2006 with four waves of 128 x 128 (25600 x
// 5120 outputs, 8192 tokens). With the loads further ahead that product takes
// 1757 to 1849 us, 1161 to 1222 TFLOP/s, of the 1380 that a large library
// product reaches on the GPU and the 1060 to 1080 it reaches in this layout.
// What bounds it is power: the matrix units are busy 59% of the cycles, at a clock
// of 1.83 GHz (of 2.4). In copies with parts left out, MFMAs and their LDS reads
// alone ran at 1650 TFLOP/s, the copies and loads cost 17 to 20% and decoding 10
// to 13%. These are times of a GPU at work: its first 40 or so launches after an
// idle time take up to a quarter longer.
template <int KIND, int EDGE>
MUON_INLINE void wgrad_tile() {
  typedef Geo<EDGE> Z;
  __shared__ __align__(1024) unsigned char smem[Z::LDS];
  constexpr int NW = Z::NW, NT = Z::NT, FM = Z::FM, NB = Z::NB;
  const ArgsPtr a = (ArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
  const int unit = xcd_unit(blockIdx.x, a->units);
  const int idx = item_of(a, unit);
  const __attribute__((address_space(4))) WgItem& it = a->item[idx];
  const int tiles = it.tiles_n * it.tiles_k;
  const int local = unit - a->unit0[idx], split = local / tiles, tile = local - split * tiles;
  int tn, tk;
  tile_of(tile, it.tiles_n, it.tiles_k, tn, tk);
  const int n0 = tn * EDGE, k0 = tk * EDGE;
  const int per_plane = (it.rows + kWgStep - 1) / kWgStep;
  const int total = per_plane * it.parts;
  // split s takes stages [total*s/splits, total*(s+1)/splits)
  const int s_begin = (int)((int64_t)total * split / it.splits);
  const int s_end = (int)((int64_t)total * (split + 1) / it.splits);

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / (NW / 2), wn = wave % (NW / 2);
  f32x16 acc[FM][NB];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
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

  // dY: instruction (wave, p) copies DMA_ROWS token rows from row DMA_ROWS*(DMA*wave
  // + p) on; of them lane l carries slot l % (EDGE/8) of row l / (EDGE/8), which
  // holds chunk slot ^ swz(row).
  // Chunks past the last column read the last one: columns are independent,
  // and those are never stored.
  uint32_t dvoff[Z::DMA];
#pragma unroll
  for (int p = 0; p < Z::DMA; ++p) {
    const int r = Z::DMA_ROWS * (Z::DMA * wave + p) + lane / (EDGE / 8);
    dvoff[p] = (uint32_t)min(r, rows - 1) * (uint32_t)(lda * 2) +
               min((lane % (EDGE / 8)) ^ lds_swizzle_k(r), (it.na - n0) / 8 - 1) * 16;
  }
  auto dy_base = [&](const Stage& g) __attribute__((always_inline)) {
    return g.dy + min(g.t0, last_base) * lda + n0;
  };
  auto copy_dy = [&](const u16* base, uint32_t buf, int p) __attribute__((always_inline)) {
    dma16s(base, dvoff[p], lds0 + buf + (wave * Z::DMA + p) * 1024);
  };
  // X: chunk c of a thread is bytes 16*(tid % ROW_CHUNKS) .. of token row ROW_STEP*c +
  // tid / ROW_CHUNKS.
  const int qr = tid / Z::ROW_CHUNKS, qc = tid % Z::ROW_CHUNKS;
  const int qcol = k0 + 16 * min(qc, (it.k - 1 - k0) / 16);  // the last chunk with a column of this matrix
  uint32_t qvoff[Z::CHUNKS], evoff[Z::CHUNKS];
#pragma unroll
  for (int c = 0; c < Z::CHUNKS; ++c) {
    const uint32_t r = (uint32_t)min(Z::ROW_STEP * c + qr, rows - 1);
    qvoff[c] = r * (uint32_t)ldq + qcol;
    evoff[c] = r * (uint32_t)lde + qcol / kGroup;
  }
  u32x4 qv[2][Z::CHUNKS], qd[Z::CHUNKS];  // two stages on their way, one being decoded
  uint32_t ev[2][Z::CHUNKS], ed[Z::CHUNKS];
  auto load_x = [&](const Stage& g, int set, int c) __attribute__((always_inline)) {
    const int64_t t = min(g.t0, last_base);
    qv[set][c] = gload16(xq + t * ldq + qvoff[c]);
    ev[set][c] = *((const g_u8*)(xe + t * lde + evoff[c]));
  };
  auto take_x = [&](int set) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < Z::CHUNKS; ++c) {
      qd[c] = qv[set][c];
      ed[c] = ev[set][c];
      asm volatile("" : "+v"(qd[c]), "+v"(ed[c]));
    }
  };
  // Bytes 4w .. 4w+3 of chunk c as bf16; w odd completes 16 bytes, which are
  // stored. Rows that are not the stage's become zeros.
  const uint32_t xoff = qr * Z::ROW, xslot = (uint32_t)(2 * qc) ^ lds_swizzle_k(qr);
  u32x4 half;
  auto write_x = [&](int skip, uint32_t buf, int c, int w) __attribute__((always_inline)) {
    const int r = Z::ROW_STEP * c + qr;
    const u32x2 t = Q8Group<KIND>(ed[c], r >= skip && r < rows).bf16x4(qd[c][w]);
    half[2 * (w & 1)] = t[0];
    half[2 * (w & 1) + 1] = t[1];
    if (w & 1)
      *reinterpret_cast<u32x4*>(smem + buf + xoff + Z::ROW_STEP * c * Z::ROW + ((xslot ^ (w >> 1)) << 4)) = half;
  };
  // A chunk whose exponent write_x cannot take is written once more. Rare, so the
  // test is all it costs, two instructions a chunk.
  auto rewrite_wide_x = [&](int skip, uint32_t buf, int c) __attribute__((always_inline)) {
    if constexpr (KIND == MUON_Q8_INT8) {
      if (__builtin_expect(ed[c] >= kQ8WideExp, 0)) {
        const int r = Z::ROW_STEP * c + qr;
        const bool live = r >= skip && r < rows;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x2 lo = q8_bf16x4_wide(qd[c][2 * h], ed[c], live), hi = q8_bf16x4_wide(qd[c][2 * h + 1], ed[c], live);
          *reinterpret_cast<u32x4*>(smem + buf + xoff + Z::ROW_STEP * c * Z::ROW + ((xslot ^ h) << 4)) =
              u32x4{lo[0], lo[1], hi[0], hi[1]};
        }
      }
    }
  };
  // Rows of dY that are not the stage's become zeros once they are in LDS.
  auto clear_dy = [&](const Stage& g, uint32_t buf) __attribute__((always_inline)) {
    const int skip = g.t0 - min(g.t0, last_base);
    if (skip == 0 && rows >= kWgStep) return;
    const u32x4 z = {0u, 0u, 0u, 0u};
    for (int o = tid * 16; o < Z::OP; o += NT * 16) {
      const int r = o / Z::ROW;
      if (r < skip || r >= rows) *reinterpret_cast<u32x4*>(smem + buf + o) = z;
    }
    __syncthreads();
  };

  // Fragments: lane group G = lane/16, lane i16 points at token row 8*(G/2) +
  // i16/4 (+4 for the upper half, +16 per sub-step) and four columns.
  const int G = lane >> 4, i16 = lane & 15;
  const uint32_t frow = (8 * (G >> 1) + (i16 >> 2)) * Z::ROW;
  uint32_t foff[2][FM];
#pragma unroll
  for (int j = 0; j < FM; ++j) {  // FM >= NB
    const int col = 32 * j + 16 * (G & 1) + 4 * (i16 & 3);
    foff[0][j] = frow + ((((wm * (EDGE / 2) + col) >> 3) ^ lds_swizzle_k(i16 >> 2)) << 4) + 8 * (i16 & 1);
    foff[1][j] = frow + ((((wn * NB * 32 + col) >> 3) ^ lds_swizzle_k(i16 >> 2)) << 4) + 8 * (i16 & 1);
  }
  bf16x8 fy[2][FM], fx[2][NB];
  // Fragment f of a sub-step, in the order in which the MFMAs need them:
  // dY block 0, the blocks of X, the other blocks of dY.
  uint32_t fat[2][FM];  // where this stage's lie
  auto frags_at = [&](uint32_t dybuf, uint32_t xbuf) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      fat[0][j] = foff[0][j] + dybuf;
      fat[1][j] = foff[1][j] + xbuf;
    }
  };
  auto read_frag = [&](int b, int kk, int f) __attribute__((always_inline)) {
    const bool is_x = f >= 1 && f <= NB;
    const int j = is_x ? f - 1 : f == 0 ? 0 : f - NB;
    const unsigned char* p = smem + fat[is_x][j] + kk * 16 * Z::ROW;
    const v4i16 lo = lds_read_tr(p), hi = lds_read_tr(p + 4 * Z::ROW);
    const bf16x8 v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    if (is_x) fx[b][j] = v;
    else fy[b][j] = v;
  };

  if (s_begin < s_end) {
    const int plane = s_begin / per_plane;
    Stage g1{static_cast<const u16*>(it.dy) + (int64_t)plane * rows * lda, (s_begin - plane * per_plane) * kWgStep};
    auto skip_of = [&](const Stage& g) { return g.t0 - min(g.t0, last_base); };
    uint32_t d0 = 0, d1 = Z::OP, d2 = 2 * Z::OP;  // dY of this stage, the next, the one after
    uint32_t x0 = Z::DY_BUFS * Z::OP, x1 = x0 + Z::OP;
#pragma unroll
    for (int c = 0; c < Z::CHUNKS; ++c) load_x(g1, 0, c);
    const u16* base = dy_base(g1);
#pragma unroll
    for (int p = 0; p < Z::DMA; ++p) copy_dy(base, d0, p);
    take_x(0);
#pragma unroll
    for (int c = 0; c < Z::CHUNKS; ++c) {
#pragma unroll
      for (int w = 0; w < 4; ++w) write_x(skip_of(g1), x0, c, w);
      rewrite_wide_x(skip_of(g1), x0, c);
    }
    // g1, g2, g3: one, two and three stages ahead of the loop's. Stages past
    // the last one are the last one again, and nothing of them is used.
    const Stage first = g1;
    if (s_begin + 1 < s_end) next(g1);
    Stage g2 = g1;
    if (s_begin + 2 < s_end) next(g2);
    Stage g3 = g2;
#pragma unroll
    for (int c = 0; c < Z::CHUNKS; ++c) load_x(g1, 0, c);
#pragma unroll
    for (int c = 0; c < Z::CHUNKS; ++c) load_x(g2, 1, c);
    base = dy_base(g1);
#pragma unroll
    for (int p = 0; p < Z::DMA; ++p) copy_dy(base, d1, p);
    wait_vmcnt<0>();
    __syncthreads();
    clear_dy(first, d0);
    frags_at(d0, x0);
#pragma unroll
    for (int f = 0; f < FM + NB; ++f) read_frag(0, 0, f);

    // One stage is SLOTS MFMAs per wave. Between two of them goes a little of
    // everything else, in a fixed order: the fragments of the next sub-step,
    // the loads of X three stages ahead and the copies of dY two ahead, and
    // the decoding of the next stage's X. The last sub-step's fragments are in
    // registers a few MFMAs before its end: there the workgroup meets, and the
    // next stage's first fragments are read under the remaining MFMAs.
    //
    // What a wave waits for is always a whole stage old. take_x() makes the
    // compiler wait for this set's loads, issued two stages ago; it counts the
    // other set's as issued since and leaves as many in flight, which are the
    // copies of the stage before (it does not know of those). The wait at the
    // meeting is for these copies; since then this wave has issued its loads
    // of X, two per chunk, and Z::DMA copies.
    constexpr int kPer = Z::PER, kMeet = Z::MEET;
    auto stage = [&](auto parity, int s) __attribute__((always_inline)) {
      constexpr int P = decltype(parity)::value;
      const int skip = skip_of(g1);
      if (s + 3 < s_end) next(g3);
      const u16* base2 = dy_base(g2);
      take_x(P);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int m = 0; m < kPer; ++m) {
          const int slot = kPer * kk + m;
          if (slot == kMeet) {
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(2 * Z::CHUNKS + Z::DMA) : "memory");
            clear_dy(g1, d1);
            frags_at(d1, x1);
          }
          const int i = m / NB, j = m % NB;
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fx[kk & 1][j], fy[kk & 1][i], acc[i][j], 0, 0, 0);
          if (kk < 3 && m < FM + NB) read_frag((kk + 1) & 1, kk + 1, m);
          if (slot >= kMeet) read_frag(0, 0, slot - kMeet);
          if (slot < 2 * Z::CHUNKS && m % 2 == 1) load_x(g3, P, m / 2);
          if (slot >= 2 * Z::CHUNKS && slot < 2 * (Z::CHUNKS + Z::DMA) && m % 2 == 1) copy_dy(base2, d2, slot / 2 - Z::CHUNKS);
          const int piece = (slot - Z::DEC0) / Z::DEC;
          if (slot >= Z::DEC0 && piece < 4 * Z::CHUNKS && (slot - Z::DEC0) % Z::DEC == 0) {
            write_x(skip, x1, piece / 4, piece % 4);
            if (piece % 4 == 3) rewrite_wide_x(skip, x1, piece / 4);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      g1 = g2;
      g2 = g3;
      const uint32_t d = d0;
      d0 = d1, d1 = d2, d2 = d;
      const uint32_t x = x0;
      x0 = x1, x1 = x;
    };
    int s = s_begin;
    for (; s + 1 < s_end; s += 2) {
      stage(std::integral_constant<int, 0>{}, s);
      stage(std::integral_constant<int, 1>{}, s + 1);
    }
    if (s < s_end) stage(std::integral_constant<int, 0>{}, s);
    wait_vmcnt<0>();  // the copies past the last stage, before this LDS is used again
    __syncthreads();
  }

  // The tile leaves through LDS in fp32 (256: in two halves, blocks 0, 1 and 2,
  // 3 of every wave), 128 rows at a time, so that a wave stores whole rows. The
  // 16-byte unit u of row r sits at unit u ^ (r % 64) (128: r % 32).
  constexpr int LW = EDGE / 4, HALVES = FM / 2, MASK = LW - 1;
  const int ftid = fresh_tid(), flane = ftid & 63;  // keeps these addresses out of the loop's registers
  const GradOut<LW, true> out(it, a, ftid % LW, k0);
#pragma unroll
  for (int half = 0; half < HALVES; ++half) {
    if (half) __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int r = wm * 64 + 32 * i + (flane & 31), u = wn * 8 * NB + 8 * j + 2 * g + (flane >> 5);
          const f32x16& t = acc[2 * half + i][j];
          *reinterpret_cast<f32x4*>(smem + r * EDGE * 4 + ((u ^ (r & MASK)) << 4)) =
              f32x4{t[4 * g], t[4 * g + 1], t[4 * g + 2], t[4 * g + 3]};
        }
    __syncthreads();
#pragma unroll 4
    for (int q = 0; q < 128 * LW / NT; ++q) {
      const int r = q * (NT / LW) + (LW == 64 ? wave : ftid / LW), n = (r >> 6) * (EDGE / 2) + half * 64 + (r & 63);
      const unsigned char* row = smem + r * EDGE * 4;
      float v[4];
      out.gather(v, [&](int u) { return reinterpret_cast<const float*>(row + ((u ^ (r & MASK)) << 4)); }, it.splits > 1);
      if (it.splits > 1) Vec4<float>::store(a->partial + ((int64_t)(it.part0 + local) * EDGE + n) * EDGE + 4 * out.lane, v);
      else out.store(n0 + n, v);
    }
  }
}

template <int KIND>
__global__ void __launch_bounds__(Geo<256>::NT, 2) wgrad_kernel(WgArgs) {
  wgrad_tile<KIND, 256>();
}

// 128 x 128 tiles, two workgroups per CU: for products with too few 256 x 256
// tiles for the CUs but long enough a sum to be bound by arithmetic, not by the
// chain of one tile. 13 to 16 us at 300 bf16 tokens, 2048 x 2048 (160 to 195
// TFLOP/s; 25 us with 256 x 256 tiles, 24 with 64 x 64), 30 at 1000 tokens, 1024 x 5120 (350
// TFLOP/s; 40 with either). A round of 512 takes 1.16 us per stage, the same
// outputs in 256 x 256 tiles half of a round's 1.4: a byte of an operand moved
// to LDS feeds half as many MFMAs, and a byte read from it two thirds.
template <int KIND>
__global__ void __launch_bounds__(Geo<128>::NT, 2) wgrad_medium_kernel(WgArgs) {
  wgrad_tile<KIND, 128>();
}

// ------------------------------------------------------------ small tiles
//
// 64 x 64 output tiles for products that would leave most CUs without a
// larger one: a call of a few small matrices is over in the time of its
// memory round trips, and what counts is how many of these it takes. Each of
// the four waves sums every fourth block of 32 tokens for the whole tile, on
// its own: it stages both operands in an LDS region that only it uses, with
// the next block's loads in flight, and nothing synchronises the workgroup
// until the four sums are added. dY is read as it is, in any alignment, and
// fp32 values are cut into their three bf16 parts on the way to LDS, so there
// is no other launch. 101 tokens, 203 x 137 outputs, fp32: 7.6 us (54 with the
// large kernel); with the GPU full it reaches about 215 TFLOP/s.

constexpr int kSmRow = kWgSmall * 2;     // bytes of an LDS row: 64 bf16 of one token
constexpr int kSmOp = 32 * kSmRow;       // one operand of 32 tokens: 4 KB

// x = hi + mid + lo, each the rest rounded toward zero to bf16: 8 bits each,
// all 24 of an fp32 number of at least 2^-110 (of smaller ones the bits down to
// 2^-133), and never past the largest finite value.
// Infinities and NaNs stay in hi alone. Returned as fp32 bit patterns whose
// low halves are zero.
MUON_INLINE void split3(float x, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  const uint32_t bits = __float_as_uint(x);
  const bool fine = (bits & 0x7f800000u) != 0x7f800000u;
  hi = fine ? bits & 0xffff0000u : __float_as_uint(bf16_to_f32(f32_to_bf16(x)));
  const float r = fine ? x - __uint_as_float(hi) : 0.f;
  mid = __float_as_uint(r) & 0xffff0000u;
  lo = __float_as_uint(r - __uint_as_float(mid)) & 0xffff0000u;
}

// Columns c0 .. c0+7 of a row of n elements at any alignment; past n, the last
// column again. Only a row's last columns are loaded one by one. Nothing here
// waits for the loads, so the caller clears what is past n later.
template <class T>
MUON_INLINE void load_dy8(const T* row, int c0, int n, float v[8]) {
  if (c0 + 8 <= n) {
    if constexpr (sizeof(T) == 4) {
      const u32x4 lo = gload16_any(row + c0), hi = gload16_any(row + c0 + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = __uint_as_float(lo[i]);
        v[4 + i] = __uint_as_float(hi[i]);
      }
    } else {
      const u32x4 w = gload16_any(row + c0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = Elem<T>::load(row + min(c0 + i, n - 1));
  }
}

// The slot of 16-byte chunk c of token row r: rows r .. r+3, which a
// transposing read takes together, lie in different banks.
MUON_INLINE int small_slot(int c, int r) { return c ^ ((r & 3) << 1); }

template <int KIND, class T>
__global__ void __launch_bounds__(256, 2) wgrad_small_kernel(WgArgs) {
  constexpr int PARTS = sizeof(T) == 4 ? 3 : 1;
  __shared__ __align__(1024) unsigned char smem[4 * 4 * kSmOp];
  const ArgsPtr a = (ArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
  const int unit = xcd_unit(blockIdx.x, a->units);
  const int idx = item_of(a, unit);
  const __attribute__((address_space(4))) WgItem& it = a->item[idx];
  const int tiles = it.tiles_n * it.tiles_k;
  const int local = unit - a->unit0[idx], split = local / tiles, tile = local - split * tiles;
  int tn, tk;
  tile_of(tile, it.tiles_n, it.tiles_k, tn, tk);
  const int n0 = tn * kWgSmall, k0 = tk * kWgSmall;
  const int rows = it.rows, blocks = (rows + 31) / 32;
  const int b_begin = (int)((int64_t)blocks * split / it.splits), b_end = (int)((int64_t)blocks * (split + 1) / it.splits);

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  unsigned char* sy = smem + wave * 4 * kSmOp;   // PARTS planes of dY
  unsigned char* sx = sy + 3 * kSmOp;

  // dY: chunk c of a lane is 8 columns of token row 8c + lane/8; X: 16 bytes of
  // token row 16c + lane/4.
  const int yr = lane >> 3, yc = (lane & 7) * 8, xr = lane >> 2, xc = k0 + 16 * min(lane & 3, (it.k - 1 - k0) / 16);
  const T* dy = static_cast<const T*>(it.dy);
  const int ycols = it.n - n0 - yc;  // of a lane's 8 columns, the ones that exist
  float yv[4][8];
  u32x4 xv[2];
  uint32_t ev[2];
  // Tokens past the last one read the last one, and become zeros when they are
  // staged.
  auto load = [&](int b) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      load_dy8(dy + (int64_t)min(32 * b + 8 * c + yr, rows - 1) * it.lda, n0 + yc, it.n, yv[c]);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int64_t t = min(32 * b + 16 * c + xr, rows - 1);
      xv[c] = gload16(it.q + t * it.ldq + xc);
      ev[c] = *((const g_u8*)(it.e + t * it.lde + xc / kGroup));
    }
  };
  auto stage = [&](int b) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int r = 8 * c + yr;
      const int live = 32 * b + r < rows ? ycols : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) yv[c][i] = i < live ? yv[c][i] : 0.f;
      u32x4 o[PARTS];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (PARTS == 1) {
          o[0][i] = pack_bf16x2(yv[c][2 * i], yv[c][2 * i + 1]);
        } else {
          uint32_t w[2][3];
          split3(yv[c][2 * i], w[0][2], w[0][1], w[0][0]);
          split3(yv[c][2 * i + 1], w[1][2], w[1][1], w[1][0]);
#pragma unroll
          for (int q = 0; q < 3; ++q) o[q][i] = (w[0][q] >> 16) | w[1][q];
        }
      }
#pragma unroll
      for (int q = 0; q < PARTS; ++q)
        *reinterpret_cast<u32x4*>(sy + q * kSmOp + r * kSmRow + (small_slot(lane & 7, r) << 4)) = o[q];
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = 16 * c + xr;
      const bool live_x = 32 * b + r < rows;
      const Q8Group<KIND> grp(ev[c], live_x);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x2 lo = grp.bf16x4(xv[c][2 * h]), hi = grp.bf16x4(xv[c][2 * h + 1]);
        if (KIND == MUON_Q8_INT8 && __builtin_expect(ev[c] >= kQ8WideExp, 0)) {
          lo = q8_bf16x4_wide(xv[c][2 * h], ev[c], live_x);
          hi = q8_bf16x4_wide(xv[c][2 * h + 1], ev[c], live_x);
        }
        *reinterpret_cast<u32x4*>(sx + r * kSmRow + (small_slot(2 * (lane & 3) + h, r) << 4)) = u32x4{lo[0], lo[1], hi[0], hi[1]};
      }
    }
  };
  // As in the large kernel, with 64 columns: block j is columns 32j ..
  const int G = lane >> 4, i16 = lane & 15;
  auto frag = [&](const unsigned char* op, int kk, int j) __attribute__((always_inline)) {
    const int r = 16 * kk + 8 * (G >> 1) + (i16 >> 2), c = 32 * j + 16 * (G & 1) + 4 * (i16 & 3);
    const unsigned char* p = op + r * kSmRow + (small_slot(c >> 3, r) << 4) + 8 * (i16 & 1);
    const v4i16 lo = lds_read_tr(p), hi = lds_read_tr(p + 4 * kSmRow);  // rows r and r + 4 share their slots
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };

  const GradOut<16> out(it, a, lane & 15, k0);  // here, so that the scale arrives during the sum
  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  int b = b_begin + wave;
  if (b < b_end) load(b);
  for (; b < b_end; b += 4) {
    stage(b);
    wave_lds_order();
    if (b + 4 < b_end) load(b + 4);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const bf16x8 x0 = frag(sx, kk, 0), x1 = frag(sx, kk, 1);
#pragma unroll
      for (int q = 0; q < PARTS; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bf16x8 y = frag(sy + q * kSmOp, kk, i);
          acc[i][0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x0, y, acc[i][0], 0, 0, 0);
          acc[i][1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x1, y, acc[i][1], 0, 0, 0);
        }
    }
    wave_lds_order();
  }

  // Every wave's sums, 16 KB each (16-byte unit u of row r at u ^ (r % 16)),
  // then added in wave order: 16 lanes a row, 16 rows at a time.
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int r = 32 * i + (lane & 31), u = 8 * j + 2 * g + (lane >> 5);
        const f32x16& t = acc[i][j];
        *reinterpret_cast<f32x4*>(sy + r * 256 + ((u ^ (r & 15)) << 4)) = f32x4{t[4 * g], t[4 * g + 1], t[4 * g + 2], t[4 * g + 3]};
      }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int r = 16 * q + (tid >> 4);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const unsigned char* row = smem + w * 4 * kSmOp + r * 256;
      float t[4];
      out.gather(t, [&](int u) { return reinterpret_cast<const float*>(row + ((u ^ (r & 15)) << 4)); }, it.splits > 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += t[i];
    }
    if (it.splits > 1)
      Vec4<float>::store(a->partial + (int64_t)(it.part0 + local) * kWgSmall * kWgSmall + r * kWgSmall + 4 * out.lane, v);
    else
      out.store(n0 + r, v);
  }
}

// ------------------------------------------------------------ joins

// Adds an item's partial tiles in split order and stores the gradient. A
// workgroup takes 1024 elements of one tile: whole rows. Bound by memory: three
// pieces of 1024 x 5120 fp32 accumulated into a gradient, 105 MB, in 19 us (5.5
// TB/s).
template <int EDGE>
__global__ void __launch_bounds__(256) wgrad_reduce_kernel(WgArgs) {
  constexpr int LW = EDGE / 4, PER = EDGE * EDGE / 1024;  // lanes per row, workgroups per tile
  const ArgsPtr a = (ArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
  // workgroups are numbered over the tiles of the items with splits
  int b = blockIdx.x, idx = 0;
  for (; idx < a->n_items; ++idx) {
    const int mine = a->item[idx].splits > 1 ? a->item[idx].tiles_n * a->item[idx].tiles_k * PER : 0;
    if (b < mine) break;
    b -= mine;
  }
  const __attribute__((address_space(4))) WgItem& it = a->item[idx];
  const int tiles = it.tiles_n * it.tiles_k, tile = b / PER;
  const int row = (b % PER) * (256 / LW) + threadIdx.x / LW;
  int tn, tk;
  tile_of(tile, it.tiles_n, it.tiles_k, tn, tk);
  const GradOut<LW> out(it, a, threadIdx.x % LW, tk * EDGE);
  const float* p = a->partial + (int64_t)(it.part0 + tile) * EDGE * EDGE + row * EDGE;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  const int64_t step = (int64_t)tiles * EDGE * EDGE;
  if (out.vec) {
#pragma unroll 4
    for (int s = 0; s < it.splits; ++s) {
      float t[4];
      Vec4<float>::load(p + s * step + 4 * out.lane, t);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += t[i];
    }
  } else {
#pragma unroll 4
    for (int s = 0; s < it.splits; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += Elem<float>::load(p + s * step + out.col(i));
  }
  out.store(tn * EDGE + row, v);
}

template <int EDGE>
static hipError_t launch_reduce(const WgArgs& args, hipStream_t s) {
  int64_t blocks = 0;
  for (int i = 0; i < args.n_items; ++i)
    if (args.item[i].splits > 1) blocks += (int64_t)args.item[i].tiles_n * args.item[i].tiles_k * (EDGE * EDGE / 1024);
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL(wgrad_reduce_kernel<EDGE>, dim3((uint32_t)blocks), dim3(256), 0, s, args);
  return hipGetLastError();
}

hipError_t launch_wgrad(const WgArgs& args, int kind, hipStream_t s) {
  const dim3 grid(args.units);
  if (args.edge == kWgTile) {
    if (kind == MUON_Q8_INT8) hipLaunchKernelGGL(wgrad_kernel<MUON_Q8_INT8>, grid, dim3(Geo<256>::NT), 0, s, args);
    else hipLaunchKernelGGL(wgrad_kernel<MUON_Q8_E4M3>, grid, dim3(Geo<256>::NT), 0, s, args);
  } else if (args.edge == kWgMedium) {
    if (kind == MUON_Q8_INT8) hipLaunchKernelGGL(wgrad_medium_kernel<MUON_Q8_INT8>, grid, dim3(Geo<128>::NT), 0, s, args);
    else hipLaunchKernelGGL(wgrad_medium_kernel<MUON_Q8_E4M3>, grid, dim3(Geo<128>::NT), 0, s, args);
  } else if (args.dy_f32) {
    if (kind == MUON_Q8_INT8) hipLaunchKernelGGL((wgrad_small_kernel<MUON_Q8_INT8, float>), grid, dim3(256), 0, s, args);
    else hipLaunchKernelGGL((wgrad_small_kernel<MUON_Q8_E4M3, float>), grid, dim3(256), 0, s, args);
  } else {
    if (kind == MUON_Q8_INT8) hipLaunchKernelGGL((wgrad_small_kernel<MUON_Q8_INT8, u16>), grid, dim3(256), 0, s, args);
    else hipLaunchKernelGGL((wgrad_small_kernel<MUON_Q8_E4M3, u16>), grid, dim3(256), 0, s, args);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return args.edge == kWgTile ? launch_reduce<kWgTile>(args, s)
         : args.edge == kWgMedium ? launch_reduce<kWgMedium>(args, s) : launch_reduce<kWgSmall>(args, s);
}

// dY in other layouts than the large kernel's (fp32, unaligned rows, a width
// that is no multiple of 8): rewritten once, as one bf16 plane or as the three
// planes lo, mid, hi of fp32 values, rows of lda columns (zeros past n). Bound by
// memory; it pays because every element is then read by many tiles.
template <class T, int PARTS>
__global__ void __launch_bounds__(256) wgrad_pack_kernel(const T* dy, int64_t ld, u16* out, int32_t rows, int32_t n,
                                                         int64_t lda) {
  const int64_t octets = lda / 8, count = octets * rows;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / octets, c0 = (i - row * octets) * 8;
    float v[8];
    load_dy8(dy + row * ld, (int)c0, n, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c0 + e < n ? v[e] : 0.f;
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
        for (int h = 0; h < 2; ++h) split3(v[2 * e + h], b[2][h], b[1][h], b[0][h]);
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
