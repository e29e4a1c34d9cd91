// Internal types shared by the host side of the layer operators
// (layer_api.cpp) and their kernels (layer_kernels.hip, wgrad_kernels.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "muon.h"

namespace muon {

constexpr int kGroup = 32;           // columns that share one exponent byte
constexpr int kNormMaxCols = 32768;  // 1024 threads x 4 x 8 columns
constexpr int kMinExp = 17;          // smallest exponent byte: 2^-110

// A norm workgroup holds one row, 8 columns per thread, `vecs` times. The
// forward kernel needs few registers and goes to 1024 threads first; the
// backward kernel's partial sums need 24 per 8 columns, so it takes at most 768
// threads (168 registers each), then 512 (256). Rows past 8192 columns do not fit
// the registers either way and spill.
inline int norm_forward_vecs(int64_t cols) { return cols <= 8192 ? 1 : cols <= 16384 ? 2 : 4; }
inline int norm_backward_vecs(int64_t cols) { return cols <= 6144 ? 1 : cols <= 8192 ? 2 : 4; }
inline int norm_threads(int64_t cols, int vecs) {
  const int64_t per = 8 * vecs;
  return int(((cols + per - 1) / per + 63) / 64 * 64);
}

// Rows of up to 512 columns are one wave each, several to a workgroup: forward
// 4; backward 8, which leave fewer partial sums (8192 x 512 bf16: 16.9 us, with
// 4 17.5, with 2 21; one row per workgroup 26).
// Few rows take a workgroup each, so that they run at once (37 x 201 fp32
// backward: 5.6 us, 8 to a workgroup 10).
constexpr int kNormRowsForward = 4, kNormRowsBackward = 8;
inline int norm_rows(int64_t rows, int threads, int most) {
  return threads == 64 ? int(std::max<int64_t>(1, std::min<int64_t>(most, rows / 256))) : 1;
}

// Workgroups of the norm kernels, which take rows in turn: as many as give a CU
// `per_cu` threads. Forward 1280, two of 640 for 5120 columns (4096 x 5120 bf16:
// 28.7 us; 1024 or 640 threads 33, 2048 36), five of 256 for 2048 (16384 x 2048
// bf16: 42.5 us, with 640 threads 53). Backward 768, which is what its registers
// allow (16384 x 2048 bf16: 80 us; 512 threads 93, 1024 100: some wait). Both were
// chosen at these widths. At others, 2^24 bf16 elements take 28 to 29 us forward
// from 512 to 5120 columns and 33 to 36 from 6144 to 8192; backward 48 to 52 us
// from 512 to 6144 columns, but 69 at 2560 and 55 at 3584 (workgroups of 5 and
// 7 waves, for 12 places in a CU).
constexpr int kNormThreadsForward = 1280, kNormThreadsBackward = 768;
inline int norm_blocks(int64_t rows, int threads, int rows_per, int per_cu) {
  return int(std::min<int64_t>((rows + rows_per - 1) / rows_per, 256 * std::max(1, per_cu / (threads * rows_per))));
}

// A launch of either kernel. The backward kernel's workgroups each leave one
// partial sum per column and weight; where one workgroup takes all rows, the
// sums are whole and the second launch is saved.
struct NormLaunch {
  int vecs, threads, rows_per, blocks;
};
inline NormLaunch norm_forward_launch(int64_t rows, int64_t cols) {
  NormLaunch l{norm_forward_vecs(cols), 0, 1, 0};
  l.threads = norm_threads(cols, l.vecs);
  l.rows_per = norm_rows(rows, l.threads, kNormRowsForward);
  l.blocks = norm_blocks(rows, l.threads, l.rows_per, kNormThreadsForward);
  return l;
}
inline NormLaunch norm_backward_launch(int64_t rows, int64_t cols) {
  NormLaunch l{norm_backward_vecs(cols), 0, 1, 0};
  l.threads = norm_threads(cols, l.vecs);
  l.rows_per = norm_rows(rows, l.threads, kNormRowsBackward);
  l.blocks = norm_blocks(rows, l.threads, l.rows_per, kNormThreadsBackward);
  return l;
}

// ------------------------------------------------------------ weight gradients

constexpr int kWgTile = 256;   // output tile edge of the large kernel
constexpr int kWgStep = 64;    // tokens per stage of it and of the medium kernel
constexpr int kWgMedium = 128; // output tile edge of the medium kernel
constexpr int kWgSmall = 64;   // output tile edge of the small kernel
constexpr int kWgItems = 16;   // matrices per launch

// One matrix of a launch. Units (tiles x splits) are numbered consecutively
// over the items.
struct WgItem {
  const void* dy;      // large and medium kernel: bf16, 16-byte aligned rows of lda elements, parts
                       // planes of `rows` rows; small kernel: the caller's
  const uint8_t* q;
  const uint8_t* e;
  const void* scale;   // dtype, or null
  void* g;
  const void* c;
  int64_t lda, ldq, lde;
  int32_t rows, n, k, na;  // na: columns of dy that may be read (a multiple of 8)
  int32_t parts;       // 1, or 3 for fp32 dY (planes of dy; the small kernel makes them itself)
  int32_t tiles_n, tiles_k;
  int32_t splits;      // > 1: partial tiles go to the workspace
  int32_t part0;       // first partial tile of this item in the workspace
  float beta;
};

struct WgArgs {
  int32_t unit0[kWgItems];  // each item's first unit; past the last item, INT32_MAX
  WgItem item[kWgItems];
  float* partial;
  int32_t n_items;
  int32_t units;
  int32_t edge;   // kWgTile, kWgMedium or kWgSmall
  int32_t dy_f32; // dtype of dY (as given) and scale
  int32_t g_f32;  // dtype of g and c
};

hipError_t launch_q8_save(const void* x, int64_t ldx, int dtype, const muon_q8& out, hipStream_t s);
hipError_t launch_q8_load(const muon_q8& in, void* x, int64_t ldx, int dtype, hipStream_t s);
hipError_t launch_norm_forward(const muon_norm_site& site, hipStream_t s);
hipError_t launch_norm_backward(const muon_norm_site& site, const muon_norm_grads& grads, hipStream_t s);
// dY (any alignment, bf16 or fp32) into `parts` bf16 planes of rows x lda.
hipError_t launch_wgrad_pack(const void* dy, int64_t ld, int dtype, void* out, int32_t rows, int32_t n, int64_t lda,
                             hipStream_t s);
hipError_t launch_wgrad(const WgArgs& args, int kind, hipStream_t s);

}  // namespace muon
