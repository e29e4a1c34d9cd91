// C ABI of the layer operators (include/muon.h): validation, the split of a
// weight gradient's work over the GPU, and the launches. Nothing is kept
// between calls.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <string>
#include <vector>

#include "layer_internal.h"
#include "muon.h"

muon_status muon_fail_message(muon_status st, const char* msg);

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30, kMaxCols = int64_t(1) << 24;
constexpr int64_t kMaxUnits = int64_t(1) << 22;  // workgroups of 512 threads in a 32-bit grid

muon_status fail(muon_status st, const std::string& msg) { return muon_fail_message(st, msg.c_str()); }
muon_status hip_status(hipError_t e) {
  if (e == hipSuccess) return MUON_OK;
  (void)hipGetLastError();
  return fail(MUON_ERR_HIP, std::string("kernel launch: ") + hipGetErrorString(e));
}

// Runs f, turning a C++ exception (out of host memory) into a status; there may
// be no memory for the message either.
template <class F>
muon_status guarded(F f) {
  try {
    return f();
  } catch (...) {
    try {
      muon_fail_message(MUON_ERR_OOM, "out of host memory");
    } catch (...) {
    }
    return MUON_ERR_OOM;
  }
}

// A strided view in bytes: row i is [base + i*pitch, base + i*pitch + width).
struct View {
  uintptr_t base;
  int64_t rows, width, pitch;
  bool written;
  const char* name;
  int item;
};

// The views of one call: checked one by one as they are added, and against each
// other by disjoint(). Empty views (no rows) take part in neither.
class Views {
 public:
  Views() { v_.reserve(32); }
  muon_status add(const void* p, int64_t rows, int64_t cols, int64_t ld, int elem, bool written, const char* name,
                  int item = -1, uintptr_t align = 0) {
    if (!p && rows > 0) return fail(MUON_ERR_INVALID_ARG, at(item) + name + " is NULL");
    if (ld < cols || ld > kMaxCols) return fail(MUON_ERR_INVALID_ARG, at(item) + name + ": row stride must be in [cols, 2^24]");
    const uintptr_t a = align ? align : uintptr_t(elem);
    if (reinterpret_cast<uintptr_t>(p) % a)
      return fail(MUON_ERR_ALIGN, at(item) + name + " is not " + std::to_string(a) + "-byte aligned");
    if (rows > 0) v_.push_back({reinterpret_cast<uintptr_t>(p), rows, cols * elem, ld * elem, written, name, item});
    return MUON_OK;
  }

  // One float per row, contiguous.
  muon_status add_floats(const float* p, int64_t rows, bool written, const char* name) {
    if (!p && rows > 0) return fail(MUON_ERR_INVALID_ARG, std::string(name) + " is NULL");
    if (reinterpret_cast<uintptr_t>(p) % 4) return fail(MUON_ERR_ALIGN, std::string(name) + " is not 4-byte aligned");
    if (rows > 0) v_.push_back({reinterpret_cast<uintptr_t>(p), 1, rows * 4, rows * 4, written, name, -1});
    return MUON_OK;
  }

  // Contiguous scratch that the call writes.
  muon_status add_range(const void* p, size_t bytes, const char* name) {
    v_.push_back({reinterpret_cast<uintptr_t>(p), 1, int64_t(bytes), int64_t(bytes), true, name, -1});
    return MUON_OK;
  }

  muon_status disjoint() {
    std::sort(v_.begin(), v_.end(), [](const View& x, const View& y) { return x.base < y.base; });
    for (size_t i = 0; i < v_.size(); ++i) {
      const uintptr_t end = v_[i].base + uintptr_t((v_[i].rows - 1) * v_[i].pitch + v_[i].width);
      for (size_t j = i + 1; j < v_.size() && v_[j].base < end; ++j)
        if ((v_[i].written || v_[j].written) && share(v_[i], v_[j]))
          return fail(MUON_ERR_ALIAS, at(v_[i].item) + v_[i].name + " overlaps " + at(v_[j].item) + v_[j].name);
    }
    return MUON_OK;
  }

  static std::string at(int item) { return item < 0 ? "" : "item " + std::to_string(item) + ": "; }

 private:
  // lo starts first and its range reaches hi's. Views of one row pitch are
  // compared by rows and columns; others count as overlapping.
  static bool share(const View& lo, const View& hi) {
    if (lo.pitch != hi.pitch) return true;
    const int64_t off = int64_t(hi.base - lo.base), dr = off / lo.pitch, dc = off % lo.pitch;
    if (dc + hi.width > lo.pitch) return true;  // hi's rows wrap into lo's next row
    return dr < lo.rows && dc < lo.width;
  }
  std::vector<View> v_;
};

#define MUON_TRY(x)                      \
  do {                                   \
    const muon_status st_ = (x);         \
    if (st_ != MUON_OK) return st_;      \
  } while (0)

muon_status check_dtype(int32_t dtype, const char* what = "dtype") {
  if (dtype != MUON_F32 && dtype != MUON_BF16)
    return fail(MUON_ERR_UNSUPPORTED, std::string(what) + " must be MUON_F32 or MUON_BF16");
  return MUON_OK;
}
int elem_of(int32_t dtype) { return dtype == MUON_BF16 ? 2 : 4; }

muon_status check_size(int64_t rows, int64_t cols, int item = -1) {
  if (rows < 0 || rows > kMaxRows) return fail(MUON_ERR_INVALID_ARG, Views::at(item) + "rows must be in [0, 2^30]");
  if (cols < 1 || cols > kMaxCols) return fail(MUON_ERR_INVALID_ARG, Views::at(item) + "cols must be in [1, 2^24]");
  return MUON_OK;
}

muon_status check_q8(Views& views, const muon_q8& p, bool written, const char* name, int item = -1) {
  MUON_TRY(check_size(p.rows, p.cols, item));
  if (p.kind != MUON_Q8_INT8 && p.kind != MUON_Q8_E4M3)
    return fail(MUON_ERR_UNSUPPORTED, Views::at(item) + name + ": kind must be MUON_Q8_INT8 or MUON_Q8_E4M3");
  if (p.ldq % 16) return fail(MUON_ERR_ALIGN, Views::at(item) + name + ": ldq must be a multiple of 16");
  // the padding up to the next multiple of 16 belongs to the view
  MUON_TRY(views.add(p.q, p.rows, (p.cols + 15) / 16 * 16, p.ldq, 1, written, name, item, 16));
  return views.add(p.e, p.rows, (p.cols + muon::kGroup - 1) / muon::kGroup, p.lde, 1, written, name, item);
}

muon_status q8_call(const void* x, int64_t ldx, int32_t dtype, const muon_q8* p, bool save, void* stream) {
  return guarded([&]() -> muon_status {
    if (!p) return fail(MUON_ERR_INVALID_ARG, "the checkpoint is NULL");
    MUON_TRY(check_dtype(dtype));
    Views v;
    MUON_TRY(check_q8(v, *p, save, "checkpoint"));
    MUON_TRY(v.add(x, p->rows, p->cols, ldx, elem_of(dtype), !save, "x"));
    MUON_TRY(v.disjoint());
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return hip_status(save ? muon::launch_q8_save(x, ldx, dtype, *p, s)
                           : muon::launch_q8_load(*p, const_cast<void*>(x), ldx, dtype, s));
  });
}

// What the forward and the backward pass of a norm site have in common.
muon_status check_site(Views& v, const muon_norm_site& s) {
  MUON_TRY(check_dtype(s.dtype));
  MUON_TRY(check_size(s.rows, s.cols));
  if (s.cols > muon::kNormMaxCols) return fail(MUON_ERR_UNSUPPORTED, "cols must be <= 32768");
  const float f[] = {s.res_scale, s.branch_scale, s.eps};
  for (float x : f)
    if (!std::isfinite(x)) return fail(MUON_ERR_INVALID_ARG, "res_scale, branch_scale and eps must be finite");
  if (s.eps < 0.f) return fail(MUON_ERR_INVALID_ARG, "eps must be >= 0");
  const int e = elem_of(s.dtype);
  MUON_TRY(v.add(s.w_pre, 1, s.cols, s.cols, e, false, "w_pre"));
  if (s.w_post) MUON_TRY(v.add(s.w_post, 1, s.cols, s.cols, e, false, "w_post"));
  if (s.gate) {
    if (s.ld_gate == 0) MUON_TRY(v.add(s.gate, 1, s.cols, s.cols, e, false, "gate"));
    else MUON_TRY(v.add(s.gate, s.rows, s.cols, s.ld_gate, e, false, "gate"));
  }
  return MUON_OK;
}

muon_status check_saved(Views& v, const muon_norm_site& s, const muon_q8& p, bool written, const char* name) {
  if (p.rows != s.rows || p.cols != s.cols)
    return fail(MUON_ERR_INVALID_ARG, std::string(name) + " must be a rows x cols checkpoint");
  return check_q8(v, p, written, name);
}

muon_status norm_forward(const muon_norm_site* site, void* stream) {
  if (!site) return fail(MUON_ERR_INVALID_ARG, "site is NULL");
  const muon_norm_site& s = *site;
  Views v;
  MUON_TRY(check_site(v, s));
  const int e = elem_of(s.dtype);
  MUON_TRY(v.add(s.branch, s.rows, s.cols, s.ld_branch, e, false, "branch"));
  MUON_TRY(v.add(s.residual, s.rows, s.cols, s.ld_residual, e, false, "residual"));
  MUON_TRY(v.add(s.y, s.rows, s.cols, s.ld_y, e, true, "y"));
  MUON_TRY(v.add(s.h, s.rows, s.cols, s.ld_h, e, true, "h"));
  if (s.rstd_y) MUON_TRY(v.add_floats(s.rstd_y, s.rows, true, "rstd_y"));
  if (s.rstd_b) MUON_TRY(v.add_floats(s.rstd_b, s.rows, true, "rstd_b"));
  if (s.u.q) MUON_TRY(check_saved(v, s, s.u, true, "u"));
  if (s.v.q) MUON_TRY(check_saved(v, s, s.v, true, "v"));
  MUON_TRY(v.disjoint());
  return hip_status(muon::launch_norm_forward(s, static_cast<hipStream_t>(stream)));
}

size_t norm_workspace(int64_t rows, int64_t cols) {
  return size_t(muon::norm_backward_launch(rows, cols).blocks) * 3 * size_t((cols + 7) / 8 * 8) * sizeof(float);
}

muon_status norm_backward(const muon_norm_site* site, const muon_norm_grads* grads, void* stream) {
  if (!site || !grads) return fail(MUON_ERR_INVALID_ARG, "site or grads is NULL");
  const muon_norm_site& s = *site;
  const muon_norm_grads& g = *grads;
  Views v;
  MUON_TRY(check_site(v, s));
  const int e = elem_of(s.dtype);
  if (g.dy) MUON_TRY(v.add(g.dy, s.rows, s.cols, g.ld_dy, e, false, "dy"));
  MUON_TRY(v.add(g.dh, s.rows, s.cols, g.ld_dh, e, false, "dh"));
  MUON_TRY(v.add_floats(s.rstd_y, s.rows, false, "rstd_y"));
  MUON_TRY(check_saved(v, s, s.u, false, "u"));
  if (s.w_post) MUON_TRY(v.add_floats(s.rstd_b, s.rows, false, "rstd_b"));
  if (s.w_post || s.gate) MUON_TRY(check_saved(v, s, s.v, false, "v"));
  MUON_TRY(v.add(g.d_residual, s.rows, s.cols, g.ld_d_residual, e, true, "d_residual"));
  MUON_TRY(v.add(g.d_branch, s.rows, s.cols, g.ld_d_branch, e, true, "d_branch"));
  if (g.d_w_pre) MUON_TRY(v.add(g.d_w_pre, 1, s.cols, s.cols, e, true, "d_w_pre"));
  if (g.d_w_post) {
    if (!s.w_post) return fail(MUON_ERR_INVALID_ARG, "d_w_post is given but the site has no w_post");
    MUON_TRY(v.add(g.d_w_post, 1, s.cols, s.cols, e, true, "d_w_post"));
  }
  if (g.d_gate) {
    if (!s.gate) return fail(MUON_ERR_INVALID_ARG, "d_gate is given but the site has no gate");
    if (s.ld_gate == 0) MUON_TRY(v.add(g.d_gate, 1, s.cols, s.cols, e, true, "d_gate"));
    else MUON_TRY(v.add(g.d_gate, s.rows, s.cols, g.ld_d_gate, e, true, "d_gate"));
  }
  const size_t need = norm_workspace(s.rows, s.cols);
  if (need) {
    if (g.workspace_bytes < need)
      return fail(MUON_ERR_INVALID_ARG, "the workspace has " + std::to_string(g.workspace_bytes) + " bytes, " +
                                            std::to_string(need) + " are needed");
    if (!g.workspace) return fail(MUON_ERR_INVALID_ARG, "workspace is NULL");
    if (reinterpret_cast<uintptr_t>(g.workspace) % 16) return fail(MUON_ERR_ALIGN, "workspace is not 16-byte aligned");
    MUON_TRY(v.add_range(g.workspace, need, "workspace"));
  }
  MUON_TRY(v.disjoint());
  return hip_status(muon::launch_norm_backward(s, g, static_cast<hipStream_t>(stream)));
}

// ------------------------------------------------------------ weight gradients

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t round256(size_t v) { return (v + 255) / 256 * 256; }

// The large and the medium kernel read dY as it is if its rows are 16-byte
// aligned bf16 with whole 16-byte chunks; otherwise it is rewritten into the
// workspace first.
bool dy_aligned(const muon_wgrad_item& it, int32_t dtype) {
  return reinterpret_cast<uintptr_t>(it.dy) % 16 == 0 && it.ld_dy * elem_of(dtype) % 16 == 0 && it.n % 8 == 0;
}

// A way to run a launch, and what it is expected to take.
struct Choice {
  int edge, splits;
  double us;
};

// Which tile edge, and how many pieces the sum over tokens is cut into, for
// items with t256, t128 and t64 tiles in all, at most `rows` tokens, and `packed`
// bytes of dY that the two larger kernels would have rewritten first. The estimates
// are in microseconds, from sweeps on one MI355X (64 x 64 to 4000 x 4000 outputs,
// 16 to 8192 tokens, bf16 and fp32, each kernel in 1 to 16 pieces; of 174 sizes,
// 95 of them not used for the fit, the pick is over 10% behind the best in two,
// 0.2% on average):
// - large kernel: rounds of one workgroup per CU, 1.4 per stage of 64 tokens
//   and 15 to fill and empty the tile;
// - medium kernel: rounds of two per CU, 1.16 per stage, or 0.72 where one per
//   CU is left, and 10;
// - small kernel: rounds of two per CU, per 128 tokens 2.4 (fp32: 3.0), or 2.0
//   (2.3) where one per CU is left, and 2.7;
// - pieces cost their partial tiles, written and read back (256, 64 or 16 KB
//   each, at 5 to 12 TB/s, as they find a place in the caches), and one more launch;
// - rewriting dY costs a launch and its bytes at about 9 TB/s (of cache).
// For bf16, small against medium against large, each in its best number of
// pieces: 1024 x 1024 and 300 tokens 13, 15, 24 us; 2048 x 2048 and 300 tokens
// 24, 16, 25; 1024 x 1024 and 8192 tokens 87, 42, 47; 2048 x 2048 and 8192
// tokens 303, 100, 89.
Choice choose(int64_t t256, int64_t t128, int64_t t64, int64_t rows, int parts, int64_t packed) {
  constexpr int64_t kCus = 256;
  const int64_t stages = ceil_div(rows, muon::kWgStep) * parts, blocks = ceil_div(rows, 128);
  // Rounds of two workgroups per CU (the last may be of one): `fixed` each, and
  // `two` (`one`) per step.
  auto rounds = [](int64_t units, double fixed, double one, double two, double steps) {
    const int64_t full = units / (2 * kCus), rest = units % (2 * kCus);
    return fixed * double(full + (rest != 0)) + steps * (double(full) * two + (rest == 0 ? 0.0 : rest <= kCus ? one : two));
  };
  const double pack = packed ? 3.0 + double(packed) * 1.1e-7 : 0.0;
  Choice best{muon::kWgTile, 1, 1e300};
  const int64_t most = std::min<int64_t>(64, std::max(stages / 2, blocks));
  for (int s = 1; s <= std::max<int64_t>(1, most); ++s) {
    if (s == 1 || s <= stages / 2) {
      double us = 2.0 + pack + double(ceil_div(t256 * s, kCus)) * (15.0 + 1.4 * double(ceil_div(stages, s)));
      if (s > 1) us += 4.0 + 0.14 * s + 0.058 * double(t256 * s);
      if (us < best.us) best = {muon::kWgTile, s, us};
      us = 2.0 + pack + rounds(t128 * s, 10.0, 0.72, 1.16, double(ceil_div(stages, s)));
      if (s > 1) us += 4.0 + 0.14 * s + 0.011 * double(t128 * s);
      if (us < best.us) best = {muon::kWgMedium, s, us};
    }
    if (s == 1 || s <= blocks) {
      double us = rounds(t64 * s, 2.7, parts == 3 ? 2.3 : 2.0, parts == 3 ? 3.0 : 2.4, double(ceil_div(blocks, s)));
      if (s > 1) us += 4.0 + 0.14 * s + 0.006 * double(t64 * s);
      if (us < best.us) best = {muon::kWgSmall, s, us};
    }
  }
  return best;
}

struct WgradPlan {
  muon::WgArgs args;
  size_t pack[muon::kWgItems];  // workspace offset of the rewritten dY, or SIZE_MAX
  size_t partial = 0, bytes = 0;
};

// The launch of items [0, n), n <= kWgItems: descriptors and workspace layout.
muon_status plan_wgrad(const muon_wgrad_item* items, int n, int32_t dtype, int32_t g_dtype, WgradPlan& p) {
  p.args = muon::WgArgs{};
  std::fill(p.args.unit0, p.args.unit0 + muon::kWgItems, INT32_MAX);
  p.args.n_items = n;
  p.args.dy_f32 = dtype == MUON_F32;
  p.args.g_f32 = g_dtype == MUON_F32;
  const int parts = dtype == MUON_F32 ? 3 : 1;
  int64_t t256 = 0, t128 = 0, t64 = 0, rows = 0, packed = 0;
  for (int i = 0; i < n; ++i) {
    const muon_wgrad_item& it = items[i];
    t256 += ceil_div(it.n, muon::kWgTile) * ceil_div(it.x.cols, muon::kWgTile);
    t128 += ceil_div(it.n, muon::kWgMedium) * ceil_div(it.x.cols, muon::kWgMedium);
    t64 += ceil_div(it.n, muon::kWgSmall) * ceil_div(it.x.cols, muon::kWgSmall);
    rows = std::max(rows, it.x.rows);
    if (dtype == MUON_F32 || !dy_aligned(it, dtype)) packed += it.x.rows * it.n * (dtype == MUON_F32 ? 10 : 4);
  }
  const Choice choice = choose(t256, t128, t64, rows, parts, packed);
  const bool large = choice.edge != muon::kWgSmall;
  p.args.edge = choice.edge;
  size_t at = 0;
  int64_t units = 0, partials = 0;
  for (int i = 0; i < n; ++i) {
    const muon_wgrad_item& it = items[i];
    muon::WgItem& d = p.args.item[i];
    d.dy = it.dy;
    d.lda = it.ld_dy;
    d.q = static_cast<const uint8_t*>(it.x.q);
    d.e = static_cast<const uint8_t*>(it.x.e);
    d.scale = it.scale;
    d.g = it.g;
    d.c = it.c;
    d.ldq = it.x.ldq;
    d.lde = it.x.lde;
    d.rows = int32_t(it.x.rows);
    d.n = int32_t(it.n);
    d.k = int32_t(it.x.cols);
    d.na = int32_t(ceil_div(it.n, 8) * 8);
    d.parts = parts;
    d.beta = it.beta;
    p.pack[i] = SIZE_MAX;
    if (large && (dtype == MUON_F32 || !dy_aligned(it, dtype))) {
      p.pack[i] = at;
      d.lda = d.na;
      at += round256(size_t(parts) * size_t(it.x.rows) * size_t(d.na) * 2);
    }
    const int64_t pieces = large ? ceil_div(d.rows, muon::kWgStep) * parts / 2 : ceil_div(d.rows, 128);
    d.tiles_n = int32_t(ceil_div(it.n, choice.edge));
    d.tiles_k = int32_t(ceil_div(it.x.cols, choice.edge));
    const int64_t t = int64_t(d.tiles_n) * d.tiles_k;
    d.splits = int32_t(std::max<int64_t>(1, std::min<int64_t>(choice.splits, pieces)));
    p.args.unit0[i] = int32_t(units);
    d.part0 = int32_t(partials);
    units += t * d.splits;
    if (d.splits > 1) partials += t * d.splits;
    if (units > kMaxUnits) return fail(MUON_ERR_INVALID_ARG, "more than 2^22 tiles in one launch");
  }
  p.args.units = int32_t(units);
  p.partial = at;
  p.bytes = at + size_t(partials) * choice.edge * choice.edge * sizeof(float);
  return MUON_OK;
}

muon_status check_wgrad(const muon_wgrad_item* items, int32_t n, int32_t dtype, int32_t g_dtype, Views& v) {
  if (!items) return fail(MUON_ERR_INVALID_ARG, "items is NULL");
  if (n < 1) return fail(MUON_ERR_INVALID_ARG, "n_items must be >= 1");
  MUON_TRY(check_dtype(dtype));
  MUON_TRY(check_dtype(g_dtype, "g_dtype"));
  const int e = elem_of(dtype), ge = elem_of(g_dtype);
  for (int32_t i = 0; i < n; ++i) {
    const muon_wgrad_item& it = items[i];
    if (it.n < 1 || it.n > kMaxCols) return fail(MUON_ERR_INVALID_ARG, Views::at(i) + "n must be in [1, 2^24]");
    MUON_TRY(check_q8(v, it.x, false, "x", i));
    if (it.x.kind != items[0].x.kind)
      return fail(MUON_ERR_INVALID_ARG, Views::at(i) + "every checkpoint of a call must have the same kind");
    MUON_TRY(v.add(it.dy, it.x.rows, it.n, it.ld_dy, e, false, "dy", i));
    if (it.scale) MUON_TRY(v.add(it.scale, 1, it.x.cols, it.x.cols, e, false, "scale", i));
    MUON_TRY(v.add(it.g, it.n, it.x.cols, it.x.cols, ge, true, "g", i, 16));
    if (!std::isfinite(it.beta)) return fail(MUON_ERR_INVALID_ARG, Views::at(i) + "beta is not finite");
    if (it.beta != 0.f && it.c != it.g) MUON_TRY(v.add(it.c, it.n, it.x.cols, it.x.cols, ge, false, "c", i, 16));
  }
  return MUON_OK;
}

// Plans of all launches, and the workspace of the largest: launches follow each
// other on one stream and share it.
muon_status plan_all(const muon_wgrad_item* items, int32_t n, int32_t dtype, int32_t g_dtype, std::vector<WgradPlan>& plans,
                     size_t* bytes) {
  *bytes = 0;
  plans.resize((n + muon::kWgItems - 1) / muon::kWgItems);
  for (size_t i = 0; i < plans.size(); ++i) {
    const int32_t first = int32_t(i) * muon::kWgItems;
    MUON_TRY(plan_wgrad(items + first, std::min(n - first, muon::kWgItems), dtype, g_dtype, plans[i]));
    *bytes = std::max(*bytes, plans[i].bytes);
  }
  return MUON_OK;
}

// The same for items that are checked first, without a workspace.
muon_status checked_plans(const muon_wgrad_item* items, int32_t n, int32_t dtype, int32_t g_dtype,
                          std::vector<WgradPlan>& plans, size_t* bytes) {
  Views v;
  MUON_TRY(check_wgrad(items, n, dtype, g_dtype, v));
  MUON_TRY(v.disjoint());
  return plan_all(items, n, dtype, g_dtype, plans, bytes);
}

muon_status wgrad(const muon_wgrad_item* items, int32_t n, int32_t dtype, int32_t g_dtype, void* ws, size_t ws_bytes,
                  void* stream) {
  Views v;
  MUON_TRY(check_wgrad(items, n, dtype, g_dtype, v));
  size_t need = 0;
  std::vector<WgradPlan> plans;
  MUON_TRY(plan_all(items, n, dtype, g_dtype, plans, &need));
  if (need) {
    if (ws_bytes < need)
      return fail(MUON_ERR_INVALID_ARG, "the workspace has " + std::to_string(ws_bytes) + " bytes, " +
                                            std::to_string(need) + " are needed");
    if (!ws) return fail(MUON_ERR_INVALID_ARG, "workspace is NULL");
    if (reinterpret_cast<uintptr_t>(ws) % 16) return fail(MUON_ERR_ALIGN, "workspace is not 16-byte aligned");
    MUON_TRY(v.add_range(ws, need, "workspace"));
  }
  MUON_TRY(v.disjoint());
  const hipStream_t s = static_cast<hipStream_t>(stream);
  for (size_t j = 0; j < plans.size(); ++j) {
    WgradPlan& p = plans[j];
    p.args.partial = reinterpret_cast<float*>(static_cast<char*>(ws) + p.partial);
    for (int i = 0; i < p.args.n_items; ++i) {
      if (p.pack[i] == SIZE_MAX) continue;
      const muon_wgrad_item& it = items[j * muon::kWgItems + i];
      void* out = static_cast<char*>(ws) + p.pack[i];
      p.args.item[i].dy = out;
      MUON_TRY(hip_status(muon::launch_wgrad_pack(it.dy, it.ld_dy, dtype, out, int32_t(it.x.rows), int32_t(it.n),
                                                  p.args.item[i].lda, s)));
    }
    MUON_TRY(hip_status(muon::launch_wgrad(p.args, items[0].x.kind, s)));
  }
  return MUON_OK;
}

}  // namespace

extern "C" {

muon_status muon_q8_save(const void* x, int64_t ldx, int32_t dtype, const muon_q8* out, void* stream) {
  return q8_call(x, ldx, dtype, out, true, stream);
}

muon_status muon_q8_load(const muon_q8* in, void* x, int64_t ldx, int32_t dtype, void* stream) {
  return q8_call(x, ldx, dtype, in, false, stream);
}

muon_status muon_norm_forward(const muon_norm_site* site, void* stream) {
  return guarded([&] { return norm_forward(site, stream); });
}

muon_status muon_norm_backward(const muon_norm_site* site, const muon_norm_grads* grads, void* stream) {
  return guarded([&] { return norm_backward(site, grads, stream); });
}

muon_status muon_norm_backward_workspace(int64_t rows, int64_t cols, size_t* bytes) {
  return guarded([&]() -> muon_status {
    if (!bytes) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
    MUON_TRY(check_size(rows, cols));
    if (cols > muon::kNormMaxCols) return fail(MUON_ERR_UNSUPPORTED, "cols must be <= 32768");
    *bytes = norm_workspace(rows, cols);
    return MUON_OK;
  });
}

muon_status muon_wgrad(const muon_wgrad_item* items, int32_t n_items, int32_t dtype, int32_t g_dtype, void* workspace,
                       size_t workspace_bytes, void* stream) {
  return guarded([&] { return wgrad(items, n_items, dtype, g_dtype, workspace, workspace_bytes, stream); });
}

muon_status muon_wgrad_workspace(const muon_wgrad_item* items, int32_t n_items, int32_t dtype, int32_t g_dtype,
                                 size_t* bytes) {
  return guarded([&]() -> muon_status {
    if (!bytes) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
    std::vector<WgradPlan> plans;
    return checked_plans(items, n_items, dtype, g_dtype, plans, bytes);
  });
}

muon_status muon_wgrad_info(const muon_wgrad_item* items, int32_t n_items, int32_t dtype, int32_t g_dtype,
                            int32_t* tile, int32_t* pieces) {
  return guarded([&]() -> muon_status {
    if (!tile || !pieces) return fail(MUON_ERR_INVALID_ARG, "tile or pieces is NULL");
    std::vector<WgradPlan> plans;
    size_t bytes;
    MUON_TRY(checked_plans(items, n_items, dtype, g_dtype, plans, &bytes));
    for (int32_t i = 0; i < n_items; ++i) {
      const muon::WgArgs& a = plans[i / muon::kWgItems].args;
      tile[i] = a.edge;
      pieces[i] = a.item[i % muon::kWgItems].splits;
    }
    return MUON_OK;
  });
}

}  // extern "C"
