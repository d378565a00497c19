// launch.h -- launches that the entry points of several source files make
// (ops.hip has them).
#ifndef MMAOPS_LAUNCH_H
#define MMAOPS_LAUNCH_H

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "plan.h"

namespace mmaops {

// Column sums of `count` rows of FP32 partial sums, to a vector of dt; with
// `two`, of two interleaved matrices (row p of matrix y starts at (2 p + y) *
// cols).  An output that is NULL is left out.
hipError_t column_sums(const float* partial, int count, int64_t cols, void* out0, void* out1,
                       int two, int dt, hipStream_t s);

// the values of a checkpoint as a matrix of dt
hipError_t restore_to(int dt, const uint8_t* codes, const uint8_t* scales, void* y, int64_t ldy,
                      int64_t rows, int64_t cols, hipStream_t s);

// x (16-bit elements) to rows of t.ld elements at y
hipError_t align_rows(const void* x, int64_t ldx, void* y, const Stored& t, hipStream_t s);

// rows of zeros (a gradient over no rows); nothing where p is NULL
hipError_t zero_rows(void* p, int64_t ld, int64_t rows, int64_t cols, int dt, hipStream_t s);

// FN<DT, PDT>(...) for the call's types
#define MMAOPS_BY_TYPES(dt, pdt, FN, ...)                                          \
  ((dt) == kFP32   ? FN<kFP32, kFP32>(__VA_ARGS__)                                 \
   : (dt) == kFP16 ? ((pdt) == kFP32 ? FN<kFP16, kFP32>(__VA_ARGS__)               \
                                     : FN<kFP16, kFP16>(__VA_ARGS__))              \
                   : ((pdt) == kFP32 ? FN<kBF16, kFP32>(__VA_ARGS__)               \
                                     : FN<kBF16, kBF16>(__VA_ARGS__)))

}  // namespace mmaops
#endif
