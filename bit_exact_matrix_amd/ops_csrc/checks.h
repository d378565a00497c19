// checks.h -- what the C entry points check of their arguments before
// anything is enqueued, and how they report a HIP error.
#ifndef MMAOPS_CHECKS_H
#define MMAOPS_CHECKS_H

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops_common.h"
#include "plan.h"

namespace mmaops {

// keeps the error's text for mma_ops_strerror; MMAEMU_ERR_HIP
int hip_fail(hipError_t e, const char* where);

// A matrix (or vector, rows = 1) as a call reads or writes it.
struct View {
  uintptr_t p;
  int64_t rows, row_bytes, ld_bytes;
  int64_t span() const { return (rows - 1) * ld_bytes + row_bytes; }
  bool any() const { return p && rows > 0 && row_bytes > 0; }
};

inline View view(const void* p, int64_t rows, int64_t cols, int64_t ld, int esz) {
  return View{(uintptr_t)p, rows, cols * esz, ld * esz};
}

// Two matrices overlap if their spans do, unless they are side by side in
// rows of the same stride (column ranges of one buffer).
inline bool overlap(const View& a, const View& b) {
  if (!a.any() || !b.any()) return false;
  const View &lo = a.p <= b.p ? a : b, &hi = a.p <= b.p ? b : a;
  if ((uintptr_t)lo.p + (uintptr_t)lo.span() <= hi.p) return false;
  if (a.rows > 1 && b.rows > 1 && a.ld_bytes == b.ld_bytes) {
    const int64_t at = (int64_t)((hi.p - lo.p) % (uintptr_t)a.ld_bytes);
    if (at >= lo.row_bytes && at + hi.row_bytes <= a.ld_bytes) return false;
  }
  return true;
}

constexpr int kMaxViews = 16;
struct Views {
  View in[kMaxViews], out[kMaxViews];
  int ni = 0, no = 0;
  void reads(const View& v) { in[ni++] = v; }
  void writes(const View& v) { out[no++] = v; }
  bool clash() const {
    for (int i = 0; i < no; ++i) {
      for (int j = 0; j < i; ++j)
        if (overlap(out[i], out[j])) return true;
      for (int j = 0; j < ni; ++j)
        if (overlap(out[i], in[j])) return true;
    }
    return false;
  }
};

// rows x cols of elements with leading dimension ld: sizes that 64-bit byte
// offsets, the kernels' 32-bit column counters and a grid of fewer than 2^32
// lanes (16 for each column, of the column sums) hold
constexpr int64_t kMaxCols = int64_t(1) << 27, kMaxRows = int64_t(1) << 40;

inline bool shape_ok(int64_t rows, int64_t cols, int64_t ld) {
  if (rows < 0 || cols < 0 || rows > kMaxRows || cols > kMaxCols) return false;
  if (rows == 0 || cols == 0) return true;
  return (ld >= cols || rows == 1) && ld >= 0 && ld <= INT64_MAX / 8 / rows;
}

inline bool param_type_ok(int dtype, int pdt) { return pdt == dtype || pdt == kFP32; }
inline bool any_type(int dt) { return dt == kFP16 || dt == kBF16 || dt == kFP32; }
inline bool half_type(int dt) { return dt == kFP16 || dt == kBF16; }

inline int64_t scale_cols(int64_t cols) { return (cols + kBlock - 1) / kBlock; }

}  // namespace mmaops
#endif
