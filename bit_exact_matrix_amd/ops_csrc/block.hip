// block.hip -- the C ABI of the gated block's operators (include/mmaops.h):
// argument checks and launches.
#include <math.h>
#include <string.h>

#include "../../include/mmaops.h"
#include "checks.h"
#include "launch.h"
#include "residual.h"

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

// ------------------------------------------------- sum into the residual
static_assert(kNormNone == MMAOPS_NORM_NONE && kNormLayer == MMAOPS_NORM_LAYER &&
                  kNormRms == MMAOPS_NORM_RMS,
              "the kernels' norms are the ABI's");

bool norm_ok(int32_t kind) { return kind >= kNormNone && kind <= kNormRms; }

// what both passes have alike
template <typename ARGS>
int join_head(const ARGS& r, DropArgs* d) {
  if (!any_type(r.dtype) || !param_type_ok(r.dtype, r.param_dtype)) return MMAEMU_ERR_DTYPE;
  if (!norm_ok(r.post) || !norm_ok(r.pre)) return MMAEMU_ERR_UNSUPPORTED;
  if (!drop_args(r.p, r.seed, r.offset, r.state, d)) return MMAEMU_ERR_UNSUPPORTED;
  return MMAEMU_OK;
}

int check_join(const mma_residual_norm_args& r, DropArgs* d) {
  const int rc = join_head(r, d);
  if (rc) return rc;
  if (r.cols < 1 || !shape_ok(r.rows, r.cols, r.ldx) || !shape_ok(r.rows, r.cols, r.ldb) ||
      !shape_ok(r.rows, r.cols, r.ldr) ||
      (r.pre != kNormNone && !shape_ok(r.rows, r.cols, r.ldh)))
    return MMAEMU_ERR_SHAPE;
  if (r.rows == 0) return MMAEMU_OK;
  if (!r.X || !r.branch || !r.R || (r.pre != kNormNone && !r.H)) return MMAEMU_ERR_NULL;
  const int e = elem_bytes(r.dtype), pe = elem_bytes(r.param_dtype);
  const void* const vectors[5] = {r.gate, r.post_weight, r.post_bias, r.pre_weight, r.pre_bias};
  float* const stats[4] = {r.post_mean, r.post_rstd, r.mean, r.rstd};
  if (!aligned(r.X, e) || !aligned(r.branch, e) || !aligned(r.R, e) || !aligned(r.H, e) ||
      !aligned(r.state, 8))
    return MMAEMU_ERR_ALIGN;
  Views v;
  v.reads(view(r.X, r.rows, r.cols, r.ldx, e));
  v.reads(view(r.branch, r.rows, r.cols, r.ldb, e));
  v.reads(view(r.state, 1, 2, 0, 8));
  for (const void* p : vectors) {
    if (!aligned(p, pe)) return MMAEMU_ERR_ALIGN;
    v.reads(view(p, 1, r.cols, 0, pe));
  }
  v.writes(view(r.R, r.rows, r.cols, r.ldr, e));
  if (r.pre != kNormNone) v.writes(view(r.H, r.rows, r.cols, r.ldh, e));
  for (const float* p : stats) {
    if (!aligned(p, 4)) return MMAEMU_ERR_ALIGN;
    v.writes(view(p, 1, r.rows, 0, 4));
  }
  return v.clash() ? MMAEMU_ERR_ALIAS : MMAEMU_OK;
}

template <int DT, int PDT>
hipError_t join_launch(const JoinArgs& a, hipStream_t s) {
  const uint32_t grid = (uint32_t)(a.rows < 2 * kCUs ? a.rows : 2 * kCUs);
  join_long_kernel<DT, PDT><<<grid, 1024, 0, s>>>(a);
  return hipGetLastError();
}

// The workspace: the groups' column sums, then the rows' means.
struct JoinPlan {
  int groups;  // 0: no column sums
  int64_t means_at, bytes;
};

JoinPlan join_plan(const mma_residual_norm_backward_args& r) {
  JoinPlan p{0, 0, 0};
  if (r.rows == 0 ||
      !(r.dgate || r.dpost_weight || r.dpost_bias || r.dpre_weight || r.dpre_bias))
    return p;
  const int64_t runs = (r.rows + 31) / 32;
  p.groups = (int)(runs < kCUs ? runs : kCUs);
  p.means_at = up256(p.groups * 4 * r.cols * 4);
  p.bytes = p.means_at + up256(r.rows * 8);
  return p;
}

int check_join_backward(const mma_residual_norm_backward_args& r, int64_t ws_bytes,
                        const void* ws, bool sizes_only, DropArgs* d) {
  const int rc = join_head(r, d);
  if (rc) return rc;
  if (r.reserved) return MMAEMU_ERR_UNSUPPORTED;
  const bool post = r.post != kNormNone, pre = r.pre != kNormNone;
  const bool branch = r.branch && (post || r.dgate);
  if (r.cols < 1 || (r.dR && !shape_ok(r.rows, r.cols, r.lddr)) ||
      (pre && (!shape_ok(r.rows, r.cols, r.lddh) || !shape_ok(r.rows, r.cols, r.ldr))) ||
      (branch && !shape_ok(r.rows, r.cols, r.ldb)) ||
      (r.dX && !shape_ok(r.rows, r.cols, r.lddx)) ||
      (r.dbranch && !shape_ok(r.rows, r.cols, r.lddb)) || !shape_ok(r.rows, r.cols, r.cols))
    return MMAEMU_ERR_SHAPE;
  if (sizes_only) return MMAEMU_OK;
  const int e = elem_bytes(r.dtype), pe = elem_bytes(r.param_dtype);
  // gradients of the vectors of a norm that is not there
  if ((!post && (r.dpost_weight || r.dpost_bias)) || (!pre && (r.dpre_weight || r.dpre_bias)))
    return MMAEMU_ERR_UNSUPPORTED;
  void* const grads[5] = {r.dgate, r.dpost_weight, r.dpost_bias, r.dpre_weight, r.dpre_bias};
  Views v;
  for (const void* p : grads) {
    if (!aligned(p, pe)) return MMAEMU_ERR_ALIGN;
    v.writes(view(p, 1, r.cols, 0, pe));
  }
  if (r.rows == 0) return v.clash() ? MMAEMU_ERR_ALIAS : MMAEMU_OK;
  if ((!pre && !r.dR) || (pre && (!r.dH || !r.R || !r.rstd)) ||
      (r.pre == kNormLayer && !r.mean) || (post && !r.post_rstd) ||
      (r.post == kNormLayer && !r.post_mean) || ((post || r.dgate) && !r.branch))
    return MMAEMU_ERR_NULL;
  if (!aligned(r.dR, e) || !aligned(r.dH, e) || !aligned(r.R, e) || !aligned(r.branch, e) ||
      !aligned(r.dX, e) || !aligned(r.dbranch, e) || !aligned(r.state, 8) ||
      (ws && !aligned(ws, 256)))
    return MMAEMU_ERR_ALIGN;
  const int64_t need = join_plan(r).bytes;
  if (need && (!ws || ws_bytes < need)) return MMAEMU_ERR_SCRATCH;
  v.reads(view(r.dR, r.rows, r.cols, r.lddr, e));
  if (pre) {
    v.reads(view(r.dH, r.rows, r.cols, r.lddh, e));
    v.reads(view(r.R, r.rows, r.cols, r.ldr, e));
  }
  if (branch) v.reads(view(r.branch, r.rows, r.cols, r.ldb, e));
  v.reads(view(r.state, 1, 2, 0, 8));
  const void* const vectors[4] = {r.gate, r.post_weight, r.post_bias, r.pre_weight};
  const float* const stats[4] = {r.post_mean, r.post_rstd, r.mean, r.rstd};
  for (const void* p : vectors) {
    if (!aligned(p, pe)) return MMAEMU_ERR_ALIGN;
    v.reads(view(p, 1, r.cols, 0, pe));
  }
  for (const float* p : stats) {
    if (!aligned(p, 4)) return MMAEMU_ERR_ALIGN;
    v.reads(view(p, 1, r.rows, 0, 4));
  }
  v.writes(view(r.dX, r.rows, r.cols, r.lddx, e));
  v.writes(view(r.dbranch, r.rows, r.cols, r.lddb, e));
  v.writes(view(need ? ws : nullptr, 1, need, 0, 1));
  return v.clash() ? MMAEMU_ERR_ALIAS : MMAEMU_OK;
}

template <int DT, int PDT>
hipError_t join_backward_launch(const JoinArgs& a, int groups, hipStream_t s) {
  const uint32_t grid = (uint32_t)(a.rows < 2 * kCUs ? a.rows : 2 * kCUs);
  join_long_dx_kernel<DT, PDT><<<grid, 1024, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !groups) return e;
  constexpr int V = kVec<DT>;
  const dim3 sums((uint32_t)((a.cols + 64 * V - 1) / (64 * V)), (uint32_t)groups);
  join_long_sums_kernel<DT, PDT><<<sums, 256, 0, s>>>(a, (a.rows + groups - 1) / groups);
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

int mma_residual_norm(const mma_residual_norm_args* args, void* hip_stream) {
  if (!args) return MMAEMU_ERR_NULL;
  const mma_residual_norm_args& r = *args;
  JoinArgs a;
  memset(&a, 0, sizeof a);
  const int rc = check_join(r, &a.drop);
  if (rc || r.rows == 0) return rc;
  a.x = r.X;
  a.ldx = r.ldx;
  a.branch = r.branch;
  a.ldb = r.ldb;
  a.gate = r.gate;
  a.post_w = r.post_weight;
  a.post_b = r.post_bias;
  a.pre_w = r.pre_weight;
  a.pre_b = r.pre_bias;
  a.r = r.R;
  a.ldr = r.ldr;
  a.h = r.H;
  a.ldh = r.ldh;
  a.post_mean = r.post == kNormLayer ? r.post_mean : nullptr;
  a.post_rstd = r.post != kNormNone ? r.post_rstd : nullptr;
  a.mean = r.pre == kNormLayer ? r.mean : nullptr;
  a.rstd = r.pre != kNormNone ? r.rstd : nullptr;
  a.rows = r.rows;
  a.cols = (int)r.cols;
  a.post = r.post;
  a.pre = r.pre;
  a.scale = r.scale;
  a.eps = r.eps;
  (void)hipGetLastError();
  const hipError_t err =
      MMAOPS_BY_TYPES(r.dtype, r.param_dtype, join_launch, a, (hipStream_t)hip_stream);
  return err == hipSuccess ? MMAEMU_OK : hip_fail(err, "mma_residual_norm launch");
}

int64_t mma_residual_norm_backward_workspace(const mma_residual_norm_backward_args* args) {
  DropArgs d;
  if (!args || check_join_backward(*args, 0, nullptr, true, &d) != MMAEMU_OK) return 0;
  return join_plan(*args).bytes;
}

int mma_residual_norm_backward(const mma_residual_norm_backward_args* args, void* workspace,
                               int64_t workspace_bytes, void* hip_stream) {
  if (!args) return MMAEMU_ERR_NULL;
  const mma_residual_norm_backward_args& r = *args;
  JoinArgs a;
  memset(&a, 0, sizeof a);
  const int rc = check_join_backward(r, workspace_bytes, workspace, false, &a.drop);
  if (rc) return rc;
  const hipStream_t s = (hipStream_t)hip_stream;
  void* const grads[5] = {r.dgate, r.dpost_weight, r.dpost_bias, r.dpre_weight, r.dpre_bias};
  (void)hipGetLastError();
  hipError_t err = hipSuccess;
  if (r.rows == 0) {  // sums over nothing
    for (void* p : grads)
      if (err == hipSuccess) err = zero_rows(p, r.cols, 1, r.cols, r.param_dtype, s);
    return err == hipSuccess ? MMAEMU_OK : hip_fail(err, "mma_residual_norm_backward launch");
  }
  const JoinPlan plan = join_plan(r);
  if (!plan.groups && !r.dX && !r.dbranch) return MMAEMU_OK;
  a.branch = r.post != kNormNone || r.dgate ? r.branch : nullptr;
  a.ldb = r.ldb;
  a.gate = r.gate;
  a.post_w = r.post_weight;
  a.post_b = r.post_bias;
  a.pre_w = r.pre_weight;
  a.r = (void*)r.R;
  a.ldr = r.ldr;
  a.post_mean = (float*)r.post_mean;
  a.post_rstd = (float*)r.post_rstd;
  a.mean = (float*)r.mean;
  a.rstd = (float*)r.rstd;
  a.rows = r.rows;
  a.cols = (int)r.cols;
  a.post = r.post;
  a.pre = r.pre;
  a.scale = r.scale;
  a.dr = r.dR;
  a.lddr = r.lddr;
  a.dh = r.dH;
  a.lddh = r.lddh;
  a.dx = r.dX;
  a.lddx = r.lddx;
  a.db = r.dbranch;
  a.lddb = r.lddb;
  if (plan.groups) {
    a.partial = (float*)workspace;
    a.means = (float*)((char*)workspace + plan.means_at);
  }
  err = MMAOPS_BY_TYPES(r.dtype, r.param_dtype, join_backward_launch, a, plan.groups, s);
  if (err == hipSuccess && plan.groups) {
    const JoinSums j{a.partial, plan.groups, r.param_dtype, r.cols, r.gate, r.post_weight,
                     r.post_bias, r.post != kNormNone, r.dgate, r.dpost_weight, r.dpost_bias,
                     r.dpre_weight, r.dpre_bias};
    join_sums_kernel<<<(uint32_t)((r.cols + 63) / 64), 1024, 0, s>>>(j);
    err = hipGetLastError();
  }
  return err == hipSuccess ? MMAEMU_OK : hip_fail(err, "mma_residual_norm_backward launch");
}

}  // extern "C"
