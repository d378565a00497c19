// block.hip -- the C ABI of the gated block's operators (include/mmaops.h):
// argument checks and launches.
#include <math.h>
#include <string.h>

#include "../../include/mmaops.h"
#include "checks.h"
#include "launch.h"
#include "random.h"

using namespace mmaops;

namespace {

// ---------------------------------------------------------------- dropout
// p as the mask has it: a threshold for 16-bit numbers.  False where p is not
// in [0, 1] (or NaN).
bool drop_args(double p, uint64_t seed, uint64_t offset, const uint64_t* state, DropArgs* d) {
  if (!(p >= 0.0 && p <= 1.0)) return false;
  d->seed = seed;
  d->offset = offset;
  d->state = state;
  d->threshold = (uint32_t)floor(65536.0 * p + 0.5);
  d->up = d->threshold == 65536 ? 0.0f : (float)(65536.0 / (65536.0 - d->threshold));
  return true;
}

template <int DT>
hipError_t dropout_launch(const void* x, int64_t ldx, const void* residual, int64_t ldr, void* y,
                          int64_t ldy, int64_t rows, int64_t cols, const DropArgs& d,
                          hipStream_t s) {
  const int64_t vecs = (cols + 7) / 8;
  int shift = 4;
  while (shift < 8 && (int64_t(1) << shift) < vecs) ++shift;
  const int64_t per = 256 >> shift, gx = (rows + per - 1) / per;
  const int64_t gy = (vecs + (int64_t(1) << shift) - 1) >> shift;
  const dim3 grid((uint32_t)(gx < (1 << 22) ? gx : (1 << 22)), (uint32_t)(gy < 256 ? gy : 256));
  dropout_kernel<DT><<<grid, 256, 0, s>>>(x, ldx, residual, ldr, y, ldy, rows, cols, d, shift);
  return hipGetLastError();
}

}  // namespace

extern "C" {

int mma_dropout(int dtype, const void* X, int64_t ldx, const void* residual, int64_t ldr, void* Y,
                int64_t ldy, int64_t rows, int64_t cols, double p, uint64_t seed, uint64_t offset,
                const uint64_t* state, void* hip_stream) {
  if (!any_type(dtype)) return MMAEMU_ERR_DTYPE;
  DropArgs d;
  if (!drop_args(p, seed, offset, state, &d)) return MMAEMU_ERR_UNSUPPORTED;
  if (!shape_ok(rows, cols, ldx) || !shape_ok(rows, cols, ldy) ||
      (residual && !shape_ok(rows, cols, ldr)))
    return MMAEMU_ERR_SHAPE;
  if (rows == 0 || cols == 0) return MMAEMU_OK;
  if (!X || !Y) return MMAEMU_ERR_NULL;
  const int e = elem_bytes(dtype);
  if (!aligned(X, e) || !aligned(residual, e) || !aligned(Y, e) || !aligned(state, 8))
    return MMAEMU_ERR_ALIGN;
  Views v;
  v.reads(view(X, rows, cols, ldx, e));
  v.reads(view(residual, rows, cols, ldr, e));
  v.reads(view(state, 1, 2, 0, 8));
  v.writes(view(Y, rows, cols, ldy, e));
  if (v.clash()) return MMAEMU_ERR_ALIAS;
  const hipStream_t s = (hipStream_t)hip_stream;
  (void)hipGetLastError();
  const hipError_t err =
      dtype == kFP16   ? dropout_launch<kFP16>(X, ldx, residual, ldr, Y, ldy, rows, cols, d, s)
      : dtype == kBF16 ? dropout_launch<kBF16>(X, ldx, residual, ldr, Y, ldy, rows, cols, d, s)
                       : dropout_launch<kFP32>(X, ldx, residual, ldr, Y, ldy, rows, cols, d, s);
  return err == hipSuccess ? MMAEMU_OK : hip_fail(err, "mma_dropout launch");
}

}  // extern "C"
