// Descriptors shared by the host side of the layers' products (product_api.cpp)
// and their kernels (mlp_kernels.hip, linear8_kernels.hip): C[m][n] = sum_k
// A[m][k] B[n][k], or B[k][n].
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "muon.h"

namespace muon {

constexpr int kPrItems = 16;   // products per launch
constexpr int kBlock = 128;    // edge of a weight's 8-bit block

// Tiles that a launch's products are cut into.
enum PrTile { kPrLarge = 0, kPrMedium = 1, kPrSmall = 2, kPrTiles = 3 };
constexpr int kPrEdge[kPrTiles] = {256, 128, 64};

// What becomes of a product.
enum PrEpilogue {
  kPrStore = 0,    // C (+ beta * another matrix), rounded
  kPrGate = 1,     // two products a, b side by side: s = act(a) * b, and checkpoints of a, b and s
  kPrGateGrad = 2  // ds, with the checkpoints of a and b: da = ds * b * act'(a), db = ds * act(a)
};

// One product of a launch. A sum may run over several pairs of matrices of the
// same shapes: a[0] b[0]^T + a[1] b[1]^T (`sums` 2), and fp32 ones over pairs of
// bf16 planes that add up to them (`parts` 3: planes lo, mid, hi, pa and pb bytes
// apart). kPrGate: b[0] and b[1] are the two projections.
struct PrItem {
  const uint8_t* a[2];
  const uint8_t* b[2];
  int64_t lda, ldb;          // bytes; 16-byte aligned rows
  int64_t pa, pb;
  const uint8_t *ea, *eb;    // 8-bit operands: exponent bytes
  int64_t lde, ldeb_n, ldeb_k;  // of A's rows; of B's blocks, along n and along k
  int32_t m, n, k;
  int32_t sums;
  int32_t tiles_m, tiles_n;
  int32_t whole;             // the first tiles are one unit each,
  int32_t splits;            // the others as many pieces of the sum, whose partial tiles go to the workspace
  int32_t part0;             // first partial tile of this item in the workspace
  int32_t stages, per;       // of a tile's sum, and of each of its pieces (some have one more)
  // kPrStore
  void* out;
  const void* c;
  int64_t ldo, ldc;
  float beta;
};

// The gated block's epilogues.
struct PrMlp {
  muon_q8 a, b, s;           // q null: not wanted (kPrGate)
  uint16_t* plane[2];        // bf16 operands of the next product: s, or da and db; null: none
  int64_t ldp, pp;           // their row stride and the distance of their planes, elements
  void* d[2];                // kPrGateGrad: da, db as the caller wants them
  int64_t ldd[2];
  int32_t act;
  int32_t reserved;
};

struct PrArgs {
  // Units are the items' whole tiles, then their pieces, each numbered over the items:
  // an item's first; past the last item INT32_MAX.
  int32_t whole0[kPrItems], piece0[kPrItems];
  PrItem item[kPrItems];
  PrMlp mlp;
  float* partial;
  int32_t n_items, wholes, pieces;
  int32_t parts;             // 1, or 3
  int32_t f32;               // dtype of out, c and d
  int32_t tile;              // PrTile
};

// A product of at most kFewRows rows (few_kernels.hip). Strides in elements.
constexpr int kFewRows = 16, kFewHalves = 2;
struct FewArgs {
  const void* a;             // m x k
  int64_t plane;             // bf16 gated block: distance of the two planes (hi, lo) that s is cut into, or 0: one
  const void* b[2];          // n x k; the two projections of the gated block
  const uint8_t *ea, *eb;    // as in PrItem
  int64_t lda, ldb, lde, ldeb_n, ldeb_k;
  int32_t m, n, k, act;
  void* out;
  const void* c;
  int64_t ldo, ldc;
  float beta;
  int32_t per;               // rows of b per workgroup (set by the launch)
};

// Rows of b per workgroup: the same share for each of 256 CUs, in as many rounds as it
// takes with at most `most`; at least 8, since lanes without a row of their own read
// another's once more.
struct FewShare {
  int64_t per, rounds;
};
inline FewShare few_share(int64_t n, int64_t most) {
  const int64_t cus = 256, rounds = (n + cus * most - 1) / (cus * most), per = (n + cus * rounds - 1) / (cus * rounds);
  return {per < 8 ? 8 : per, rounds};
}
constexpr int kFewMost = 32, kFewMostF32 = 16;  // fp32's three parts need the registers

static_assert(sizeof(PrArgs) <= 4000, "kernel arguments");

// Operands rewritten into aligned bf16 rows (pad8 columns, zeros behind the last one),
// one plane or, of fp32, the three planes lo, mid and hi.
constexpr int kPrPacks = 4;
struct PrPack {
  const void* src;
  void* dst;
  int64_t ld, octets;        // source row stride; octets of columns of a row
  int32_t rows, cols;
  int32_t first;             // workgroup
  int32_t reserved;
};
struct PrPacks {
  PrPack pack[kPrPacks];
  int32_t n, blocks;
};

hipError_t launch_packs(const PrPacks& args, bool f32, hipStream_t s);
hipError_t launch_mlp(const PrArgs& args, int epilogue, bool transposed_b, hipStream_t s);
hipError_t launch_few(const FewArgs& args, bool f32, int ops, hipStream_t s);
hipError_t launch_few8(const FewArgs& args, hipStream_t s);
hipError_t launch_linear8(const PrArgs& args, hipStream_t s);
hipError_t launch_w8_save(const void* w, int64_t ldw, int dtype, const muon_w8& out, hipStream_t s);
hipError_t launch_w8_load(const muon_w8& in, void* w, int64_t ldw, int dtype, hipStream_t s);

}  // namespace muon
