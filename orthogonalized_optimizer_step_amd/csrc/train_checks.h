// Argument checks that the C entry points of the training-step operators share:
// views of matrix arguments, overlaps, workspaces.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <exception>
#include <string>

#include "../../include/dion.h"
#include "train_internal.h"

namespace dion {

namespace {

[[maybe_unused]] bool valid_dtype(int dtype) { return dtype == DION_BF16 || dtype == DION_FP32 || dtype == DION_FP16; }
[[maybe_unused]] int64_t esize(int dtype) { return dtype == DION_FP32 ? 4 : 2; }

// No C++ exception leaves a C entry point.
template <typename F> int guarded(F&& f) noexcept {
  try {
    return f();
  } catch (const std::exception& e) {
    try {
      return set_error(DION_E_INVAL, e.what());
    } catch (...) {
      return DION_E_INVAL;
    }
  }
}

struct Check {
  int code = DION_OK;
  std::string msg;
  void fail(int c, const std::string& m) {
    if (code == DION_OK) {
      code = c;
      msg = m;
    }
  }
  void need(bool ok, const char* m) {
    if (!ok) fail(DION_E_INVAL, m);
  }
  int done() const { return code == DION_OK ? DION_OK : set_error(code, msg); }
};

// A matrix argument in memory: rows x cols elements, ld elements from row to row.
struct View {
  const void* p;
  int64_t ld, rows, cols, es;
  const char* name;
  bool any() const { return p && rows > 0 && cols > 0; }
  const char* lo() const { return (const char*)p; }
  const char* hi() const { return lo() + ((rows - 1) * ld + cols) * es; }
};

void check_view(Check& c, const View& v) {
  if (v.rows == 0 || v.cols == 0) return;
  if (!v.p) return c.fail(DION_E_INVAL, std::string(v.name) + " is NULL");
  if ((uintptr_t)v.p % v.es) c.fail(DION_E_INVAL, std::string(v.name) + " is not aligned to its elements");
  if (v.ld < v.cols) c.fail(DION_E_INVAL, std::string(v.name) + ": rows overlap (stride below the row length)");
  if (v.rows > 1 && v.ld > INT64_MAX / 8 / v.rows) c.fail(DION_E_INVAL, std::string(v.name) + ": stride too large");
}

// `out` must not overlap `in`; with `in_place` it may be the same matrix.
void check_apart(Check& c, const View& out, const View& in, bool in_place = false) {
  if (c.code != DION_OK || !out.any() || !in.any()) return;
  if (in_place && out.p == in.p && out.es == in.es && (out.ld == in.ld || out.rows == 1)) return;
  if (out.lo() < in.hi() && in.lo() < out.hi())
    c.fail(DION_E_INVAL, std::string(out.name) + " must not overlap " + in.name);
}

void check_workspace(Check& c, const void* ws, size_t have, size_t need) {
  if (c.code != DION_OK) return;
  if (!ws) return c.fail(DION_E_WORKSPACE, "workspace is NULL");
  if ((uintptr_t)ws % 256) c.fail(DION_E_WORKSPACE, "workspace must be 256-byte aligned");
  if (have < need)
    c.fail(DION_E_WORKSPACE, "workspace too small: " + std::to_string(need) + " bytes needed, " +
                                 std::to_string(have) + " given");
}

constexpr int64_t kMaxRows = (int64_t)1 << 40;   // more than any memory holds; sizes stay far from overflow

void check_rows(Check& c, int64_t rows, int32_t cols, const char* what) {
  c.need(rows >= 0, "rows must not be negative");
  c.need(cols > 0, what);
  if (rows > kMaxRows) c.fail(DION_E_UNSUPPORTED, "more than 2^40 rows");
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// The size that an entry point reports for `scratch` bytes: kNone where it uses
// none, and more than that for any that it does use, however little.
constexpr size_t kNone = 256;
size_t reported_size(size_t scratch) { return scratch ? std::max(2 * kNone, align256(scratch)) : kNone; }

}  // namespace

}  // namespace dion
