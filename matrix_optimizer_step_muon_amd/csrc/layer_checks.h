// What the C entry points of the layer operators share (host): messages, the
// guard against exceptions, and the checks of views, sizes and checkpoints.
#pragma once

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

namespace muon {
namespace abi {

constexpr int64_t kMaxRows = int64_t(1) << 30, kMaxCols = int64_t(1) << 24;

inline muon_status fail(muon_status st, const std::string& msg) { return muon_fail_message(st, msg.c_str()); }
inline muon_status hip_status(hipError_t e) {
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

inline muon_status check_dtype(int32_t dtype, const char* what = "dtype") {
  if (dtype != MUON_F32 && dtype != MUON_BF16)
    return fail(MUON_ERR_UNSUPPORTED, std::string(what) + " must be MUON_F32 or MUON_BF16");
  return MUON_OK;
}
inline int elem_of(int32_t dtype) { return dtype == MUON_BF16 ? 2 : 4; }

inline muon_status check_size(int64_t rows, int64_t cols, int item = -1) {
  if (rows < 0 || rows > kMaxRows) return fail(MUON_ERR_INVALID_ARG, Views::at(item) + "rows must be in [0, 2^30]");
  if (cols < 1 || cols > kMaxCols) return fail(MUON_ERR_INVALID_ARG, Views::at(item) + "cols must be in [1, 2^24]");
  return MUON_OK;
}

inline muon_status check_q8(Views& views, const muon_q8& p, bool written, const char* name, int item = -1) {
  MUON_TRY(check_size(p.rows, p.cols, item));
  if (p.kind != MUON_Q8_INT8 && p.kind != MUON_Q8_E4M3)
    return fail(MUON_ERR_UNSUPPORTED, Views::at(item) + name + ": kind must be MUON_Q8_INT8 or MUON_Q8_E4M3");
  if (p.ldq % 16) return fail(MUON_ERR_ALIGN, Views::at(item) + name + ": ldq must be a multiple of 16");
  // the padding up to the next multiple of 16 belongs to the view
  MUON_TRY(views.add(p.q, p.rows, (p.cols + 15) / 16 * 16, p.ldq, 1, written, name, item, 16));
  return views.add(p.e, p.rows, (p.cols + muon::kGroup - 1) / muon::kGroup, p.lde, 1, written, name, item);
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t round256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace abi
}  // namespace muon
