// ops.hip -- the C ABI of the native training operators (include/mmaops.h):
// argument checks, the choice of kernels, and the layer norm, checkpoint
// and activation-gradient kernels.
#include <stdio.h>
#include <string.h>

#include "../../include/mmaops.h"
#include "checks.h"
#include "launch.h"
#include "linear.h"
#include "norm.h"
#include "plan.h"
#include "saved.h"

using namespace mmaops;

namespace {

static_assert(kFP16 == MMAEMU_DTYPE_FP16 && kBF16 == MMAEMU_DTYPE_BF16 &&
                  kFP32 == MMAOPS_DTYPE_FP32,
              "the kernels' type numbers are the ABI's");

thread_local char g_hip_error[256] = "no HIP error recorded";

}  // namespace

int mmaops::hip_fail(hipError_t e, const char* where) {
  snprintf(g_hip_error, sizeof g_hip_error, "HIP error in %s: %s", where, hipGetErrorString(e));
  return MMAEMU_ERR_HIP;
}

namespace {

// ------------------------------------------------------------ layer norm
// How a row is held: lanes a row, vectors a lane, rows a workgroup.
struct NormPlan {
  int gt, nv;  // gt = 0: the row is too long for registers
};

// One vector a lane and as many waves as the row needs, up to 1024 lanes;
// then two.
NormPlan norm_plan(int64_t cols, int V) {
  const int64_t vecs = (cols + V - 1) / V;
  int gt = 64;
  while (gt < 1024 && gt < vecs) gt *= 2;
  if (vecs <= gt) return {gt, 1};
  if (vecs <= 2048) return {1024, 2};
  return {0, 0};
}

// Workgroups of a row's lanes (four rows of one wave), as many as the CUs
// hold at once.
template <int DT, int PDT, int GT, int NV>
void norm_run(const NormArgs& a, hipStream_t s) {
  constexpr int G = GT == 64 ? 4 : 1;
  const int64_t groups = (a.rows + G - 1) / G;
  constexpr int kPerCU = 2048 / (GT * G);
  const uint32_t grid = (uint32_t)(groups < kCUs * kPerCU ? groups : kCUs * kPerCU);
  if (a.codes_out)
    norm_kernel<DT, PDT, GT, NV, G, true><<<grid, GT * G, 0, s>>>(a);
  else
    norm_kernel<DT, PDT, GT, NV, G, false><<<grid, GT * G, 0, s>>>(a);
}

template <int DT, int PDT>
hipError_t norm_launch(const NormArgs& a, hipStream_t s) {
  const NormPlan p = norm_plan(a.cols, kVec<DT>);
  switch (p.gt * p.nv) {
    case 64: norm_run<DT, PDT, 64, 1>(a, s); break;
    case 128: norm_run<DT, PDT, 128, 1>(a, s); break;
    case 256: norm_run<DT, PDT, 256, 1>(a, s); break;
    case 512: norm_run<DT, PDT, 512, 1>(a, s); break;
    case 1024: norm_run<DT, PDT, 1024, 1>(a, s); break;
    case 2048: norm_run<DT, PDT, 1024, 2>(a, s); break;
    default: {
      const uint32_t grid = (uint32_t)(a.rows < 2 * kCUs ? a.rows : 2 * kCUs);
      if (a.codes_out)
        norm_long_kernel<DT, true><<<grid, 1024, 0, s>>>(a, PDT);
      else
        norm_long_kernel<DT, false><<<grid, 1024, 0, s>>>(a, PDT);
    }
  }
  return hipGetLastError();
}

// Backward: workgroups of 1024 lanes, one for each CU at most, so that the
// partial sums stay at one row for each CU; rows of more than 1024 vectors
// go to the kernels that read them in several passes.
int norm_backward_groups(int64_t rows, int64_t cols, int V) {
  const NormPlan p = norm_plan(cols, V);
  if (p.gt * p.nv == 0 || p.nv > 1) {  // runs of rows of the column pass
    const int64_t runs = (rows + 31) / 32;
    return (int)(runs < kCUs ? runs : kCUs);
  }
  const int64_t g = 1024 / p.gt, groups = (rows + g - 1) / g;
  return (int)(groups < kCUs ? groups : kCUs);
}

template <int DT, int PDT, int GT>
void norm_backward_run(const NormArgs& a, int grid, hipStream_t s) {
  if (a.codes)
    norm_backward_kernel<DT, PDT, GT, 1, 1024 / GT, true><<<grid, 1024, 0, s>>>(a);
  else
    norm_backward_kernel<DT, PDT, GT, 1, 1024 / GT, false><<<grid, 1024, 0, s>>>(a);
}

template <int DT, bool SAVED>
hipError_t norm_backward_long(const NormArgs& a, int pdt, int groups, hipStream_t s) {
  if (a.partial) {  // first: dx may be written over dy
    const int V = kVec<DT>;
    const dim3 grid((uint32_t)((a.cols + 64 * V - 1) / (64 * V)), (uint32_t)groups);
    norm_long_dw_kernel<DT, SAVED><<<grid, 256, 0, s>>>(a, (a.rows + groups - 1) / groups);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.y) return e;
  }
  const uint32_t grid = (uint32_t)(a.rows < 2 * kCUs ? a.rows : 2 * kCUs);
  norm_long_dx_kernel<DT, SAVED><<<grid, 1024, 0, s>>>(a, pdt);
  return hipGetLastError();
}

template <int DT, int PDT>
hipError_t norm_backward_launch(const NormArgs& a, int groups, hipStream_t s) {
  const NormPlan p = norm_plan(a.cols, kVec<DT>);
  switch (p.gt * p.nv) {
    case 64: norm_backward_run<DT, PDT, 64>(a, groups, s); break;
    case 128: norm_backward_run<DT, PDT, 128>(a, groups, s); break;
    case 256: norm_backward_run<DT, PDT, 256>(a, groups, s); break;
    case 512: norm_backward_run<DT, PDT, 512>(a, groups, s); break;
    case 1024: norm_backward_run<DT, PDT, 1024>(a, groups, s); break;
    default:
      return a.codes ? norm_backward_long<DT, true>(a, PDT, groups, s)
                     : norm_backward_long<DT, false>(a, PDT, groups, s);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t mmaops::column_sums(const float* partial, int count, int64_t cols, void* out0,
                               void* out1, int two, int dt, hipStream_t s) {
  const dim3 grid((uint32_t)((cols + 63) / 64), two ? 2u : 1u);
  column_sum_kernel<<<grid, 1024, 0, s>>>(partial, count, cols, out0, out1, dt);
  return hipGetLastError();
}

namespace {

// ------------------------------------------------------------ checkpoints
// Lanes a row (a power of two from 16 to 256, as a shift) and the grid.
template <int DT>
void row_grid(int64_t rows, int64_t cols, int* shift, dim3* grid) {
  const int64_t vecs = scale_cols(cols) * (kBlock / kVec<DT>);
  int sh = 4;
  while (sh < 8 && (int64_t(1) << sh) < vecs) ++sh;
  const int64_t per = 256 >> sh, gx = (rows + per - 1) / per;
  const int64_t gy = (vecs + (int64_t(1) << sh) - 1) >> sh;
  *shift = sh;
  *grid = dim3((uint32_t)(gx < (1 << 22) ? gx : (1 << 22)), (uint32_t)(gy < 256 ? gy : 256));
}

template <int DT>
hipError_t save_launch(const void* x, int64_t ldx, uint8_t* codes, uint8_t* scales,
                       int64_t rows, int64_t cols, hipStream_t s) {
  int shift;
  dim3 grid;
  row_grid<DT>(rows, cols, &shift, &grid);
  save_kernel<DT><<<grid, 256, 0, s>>>(x, ldx, codes, scales, rows, cols, shift);
  return hipGetLastError();
}

template <int DT>
hipError_t restore_launch(const uint8_t* codes, const uint8_t* scales, void* y, int64_t ldy,
                          int64_t rows, int64_t cols, hipStream_t s) {
  int shift;
  dim3 grid;
  row_grid<DT>(rows, cols, &shift, &grid);
  restore_kernel<DT><<<grid, 256, 0, s>>>(codes, scales, y, ldy, rows, cols, shift);
  return hipGetLastError();
}

}  // namespace

hipError_t mmaops::restore_to(int dt, const uint8_t* codes, const uint8_t* scales, void* y,
                              int64_t ldy, int64_t rows, int64_t cols, hipStream_t s) {
  return dt == kFP16   ? restore_launch<kFP16>(codes, scales, y, ldy, rows, cols, s)
         : dt == kBF16 ? restore_launch<kBF16>(codes, scales, y, ldy, rows, cols, s)
                       : restore_launch<kFP32>(codes, scales, y, ldy, rows, cols, s);
}

// ---------------------------------------------------------------- products
// x (16-bit elements) to rows of t.ld elements at y
hipError_t mmaops::align_rows(const void* x, int64_t ldx, void* y, const Stored& t,
                              hipStream_t s) {
  if (t.rows == 0 || t.cols == 0) return hipSuccess;
  int shift;
  dim3 grid;
  row_grid<kBF16>(t.rows, t.cols, &shift, &grid);
  align_kernel<<<grid, 256, 0, s>>>((const uint16_t*)x, ldx, (uint16_t*)y, t.ld, t.rows, t.cols,
                                    shift);
  return hipGetLastError();
}

namespace {

// A product's arguments, with its operands copied where the plan says so.
hipError_t linear_fill(const Product& p, const Plan& q, LinearArgs& g, void* ws,
                       hipStream_t s) {
  const TileShape& t = kTileShape[q.tile];
  g.a = p.a;
  g.b = p.b;
  g.lda = p.lda;
  g.ldb = p.ldb;
  char* at = (char*)ws + partial_bytes(p, q);
  if (q.copy_a) {
    const Stored t = stored(p.la, p.M, p.K);
    const hipError_t e = align_rows(p.a, p.lda, at, t, s);
    if (e != hipSuccess) return e;
    g.a = at;
    g.lda = t.ld;
    at += copy_bytes(true, t);
  }
  if (q.copy_b) {
    const Stored t = stored(p.lb, p.N, p.K);
    const hipError_t e = align_rows(p.b, p.ldb, at, t, s);
    if (e != hipSuccess) return e;
    g.b = at;
    g.ldb = t.ld;
  }
  g.M = p.M;
  g.N = p.N;
  g.K = p.K;
  g.splits = q.splits;
  g.guard = q.guard;
  g.tiles_m = (int)((p.M + t.bm - 1) / t.bm);
  g.tiles_n = (int)((p.N + t.bn - 1) / t.bn);
  g.partial = q.partial ? (float*)ws : nullptr;
  return hipSuccess;
}

hipError_t linear_run(int dt, const Product& p, const Plan& q, LinearArgs g, void* ws,
                      hipStream_t s) {
  const hipError_t e = linear_fill(p, q, g, ws, s);
  if (e != hipSuccess) return e;
  return dt == kFP16 ? linear_launch_fp16(q.tile, q.direct, p.la, p.lb, g, s)
                     : linear_launch_bf16(q.tile, q.direct, p.la, p.lb, g, s);
}

// sizes whose products and tile counts the 64-bit and 31-bit counters hold
bool product_shape_ok(int64_t M, int64_t N, int64_t K) {
  constexpr int64_t kMax = kMaxCols;
  if (M < 0 || N < 0 || K < 0 || M > kMax || N > kMax || K > kMax) return false;
  return ((M + 15) / 16) * ((N + 15) / 16) <= INT32_MAX &&
         ((M + 15) / 16) * ((K + 15) / 16) <= INT32_MAX &&
         ((N + 15) / 16) * ((K + 15) / 16) <= INT32_MAX;
}

Product forward_product(const mma_linear_args& r) {
  return Product{r.M, r.N, r.K, 0, r.w_transposed ? 0 : 1, r.X, r.W, r.ldx, r.ldw};
}

int64_t linear_need(const mma_linear_args& r) {
  if (r.M == 0 || r.N == 0) return 0;
  const Product p = forward_product(r);
  return product_bytes(p, linear_plan(p, r.codes != nullptr));
}

int check_linear(const mma_linear_args& r, int64_t ws_bytes, const void* ws, bool sizes_only) {
  if (!half_type(r.dtype)) return MMAEMU_ERR_DTYPE;
  if (!param_type_ok(r.dtype, r.out_dtype) || !param_type_ok(r.dtype, r.bias_dtype))
    return MMAEMU_ERR_DTYPE;
  if (r.activation < MMAOPS_ACT_NONE || r.activation > MMAOPS_ACT_SILU || r.reserved ||
      (r.w_transposed & ~1))
    return MMAEMU_ERR_UNSUPPORTED;
  if (!product_shape_ok(r.M, r.N, r.K)) return MMAEMU_ERR_SHAPE;
  if (sizes_only) return MMAEMU_OK;
  const int64_t wr = r.w_transposed ? r.N : r.K, wc = r.w_transposed ? r.K : r.N;
  if (!shape_ok(r.M, r.K, r.ldx) || !shape_ok(wr, wc, r.ldw) || !shape_ok(r.M, r.N, r.ldy) ||
      (r.residual && !shape_ok(r.M, r.N, r.ldr)) || (r.Z && !shape_ok(r.M, r.N, r.ldz)))
    return MMAEMU_ERR_SHAPE;
  if (r.M == 0 || r.N == 0) return MMAEMU_OK;
  if (!r.Y || (r.K && (!r.X || !r.W)) || !r.codes != !r.scales) return MMAEMU_ERR_NULL;
  const int oe = elem_bytes(r.out_dtype), be = elem_bytes(r.bias_dtype);
  if (!aligned(r.X, 2) || !aligned(r.W, 2) || !aligned(r.Z, 2) || !aligned(r.Y, oe) ||
      !aligned(r.residual, oe) || !aligned(r.bias, be) || (ws && !aligned(ws, 256)))
    return MMAEMU_ERR_ALIGN;
  const int64_t need = linear_need(r);
  if (need && (!ws || ws_bytes < need)) return MMAEMU_ERR_SCRATCH;
  Views v;
  if (r.K) {
    v.reads(view(r.X, r.M, r.K, r.ldx, 2));
    v.reads(view(r.W, wr, wc, r.ldw, 2));
  }
  v.reads(view(r.bias, 1, r.N, r.N, be));
  v.reads(view(r.residual, r.M, r.N, r.ldr, oe));
  v.writes(view(r.Y, r.M, r.N, r.ldy, oe));
  v.writes(view(r.Z, r.M, r.N, r.ldz, 2));
  v.writes(view(r.codes, 1, r.M * r.N, r.M * r.N, 1));
  v.writes(view(r.scales, 1, r.M * scale_cols(r.N), 0, 1));
  v.writes(view(need ? ws : nullptr, 1, need, need, 1));
  return v.clash() ? MMAEMU_ERR_ALIAS : MMAEMU_OK;
}

// The backward pass: what it needs of the workspace, piece by piece.
struct BackwardPlan {
  Product dx, dw;
  Plan pdx, pdw;
  bool has_dz;      // dz is written (an activation, and a product to use it)
  int db_runs;      // rows of column sums, 0: no bias gradient
  int64_t db_run;   // rows of one of them
  int64_t dz_at, x_at, db_at, part_at, part2_at, bytes;
  bool pair;        // both products and the column sums in one launch
};

BackwardPlan backward_plan(const mma_linear_backward_args& r, void* ws) {
  BackwardPlan b;
  memset(&b, 0, sizeof b);
  char* const base = (char*)ws;
  int64_t at = 0;
  b.has_dz = r.activation != MMAOPS_ACT_NONE && (r.dX || r.dW);
  if (b.has_dz) {
    b.dz_at = at;
    // rows that start on 16 bytes, so that the products' loads are direct
    at += up256(r.M * ((r.N + 7) / 8 * 8) * 2);
  }
  if (r.x_codes && r.dW) {
    b.x_at = at;
    at += up256(r.M * ((r.K + 7) / 8 * 8) * 2);
  }
  if (r.dbias) {
    const int64_t cols = (r.N + 511) / 512;
    int64_t runs = (8 * kCUs + cols - 1) / cols;
    if (runs > (r.M + 7) / 8) runs = (r.M + 7) / 8;
    b.db_run = (r.M + runs - 1) / runs;
    b.db_runs = (int)((r.M + b.db_run - 1) / b.db_run);
    b.db_at = at;
    at += up256((int64_t)b.db_runs * r.N * 4);
  }
  const void* const dz = b.has_dz ? base + b.dz_at : r.dY;
  const int64_t lddz = b.has_dz ? (r.N + 7) / 8 * 8 : r.lddy;
  const void* const x = r.x_codes ? base + b.x_at : r.X;
  const int64_t ldx = r.x_codes ? (r.K + 7) / 8 * 8 : r.ldx;
  b.part_at = at;
  int64_t part = 0;
  if (r.dX) {
    b.dx = Product{r.M, r.K, r.N, 0, r.w_transposed ? 1 : 0, dz, r.W, lddz, r.ldw};
    b.pdx = linear_plan(b.dx, false);
    part = product_bytes(b.dx, b.pdx);
  }
  if (r.dW) {
    b.dw = r.w_transposed ? Product{r.N, r.K, r.M, 1, 1, dz, x, lddz, ldx}
                          : Product{r.K, r.N, r.M, 1, 1, x, dz, ldx, lddz};
    b.pdw = linear_plan(b.dw, false);
    const int64_t w = product_bytes(b.dw, b.pdw);
    part = part > w ? part : w;
  }
  // Both on small tiles, whole, and few enough that one grid holds them: one
  // launch.  Their copies, if any, then stand in the workspace side by side.
  auto tiles = [](const Product& p) { return ((p.M + 63) / 64) * ((p.N + 63) / 64); };
  b.pair = r.dX && r.dW && r.K && b.pdx.tile == kTileSmall && b.pdw.tile == kTileSmall &&
           !b.pdx.partial && !b.pdw.partial && tiles(b.dx) + tiles(b.dw) <= (1 << 20);
  b.part2_at = b.pair ? at + product_bytes(b.dx, b.pdx) : at;
  b.bytes = b.pair ? b.part2_at + product_bytes(b.dw, b.pdw) : at + part;
  return b;
}

int check_backward(const mma_linear_backward_args& r, int64_t ws_bytes, void* ws,
                   bool sizes_only) {
  if (!half_type(r.dtype)) return MMAEMU_ERR_DTYPE;
  if (!param_type_ok(r.dtype, r.dw_dtype) || !param_type_ok(r.dtype, r.bias_dtype))
    return MMAEMU_ERR_DTYPE;
  if (r.activation < MMAOPS_ACT_NONE || r.activation > MMAOPS_ACT_SILU || r.reserved ||
      (r.w_transposed & ~1))
    return MMAEMU_ERR_UNSUPPORTED;
  if (!product_shape_ok(r.M, r.N, r.K)) return MMAEMU_ERR_SHAPE;
  if (sizes_only) return MMAEMU_OK;
  const int64_t wr = r.w_transposed ? r.N : r.K, wc = r.w_transposed ? r.K : r.N;
  const bool act = r.activation != MMAOPS_ACT_NONE;
  if (!shape_ok(r.M, r.N, r.lddy) || (r.X && !shape_ok(r.M, r.K, r.ldx)) ||
      (r.dX && !shape_ok(wr, wc, r.ldw)) || (act && r.Z && !shape_ok(r.M, r.N, r.ldz)) ||
      (r.dX && !shape_ok(r.M, r.K, r.lddx)) || (r.dW && !shape_ok(wr, wc, r.lddw)))
    return MMAEMU_ERR_SHAPE;
  const bool any_dx = r.dX && r.M && r.K, any_dw = r.dW && r.K && r.N, any_db = r.dbias && r.N;
  if (!any_dx && !any_dw && !any_db) return MMAEMU_OK;
  if (r.M && r.N) {
    if (!r.dY || (any_dx && !r.W)) return MMAEMU_ERR_NULL;
    if (!r.x_codes != !r.x_scales || !r.z_codes != !r.z_scales) return MMAEMU_ERR_NULL;
    if (any_dw && !r.X == !r.x_codes) return MMAEMU_ERR_NULL;
    if (act && !r.Z == !r.z_codes) return MMAEMU_ERR_NULL;
  }
  if (!aligned(r.dY, 2) || !aligned(r.X, 2) || !aligned(r.W, 2) || !aligned(r.Z, 2) ||
      !aligned(r.dX, 2) || !aligned(r.dW, elem_bytes(r.dw_dtype)) ||
      !aligned(r.dbias, elem_bytes(r.bias_dtype)) || (ws && !aligned(ws, 256)))
    return MMAEMU_ERR_ALIGN;
  const int64_t need = r.M && r.N ? backward_plan(r, ws).bytes : 0;
  if (need && (!ws || ws_bytes < need)) return MMAEMU_ERR_SCRATCH;
  Views v;
  v.reads(view(r.dY, r.M, r.N, r.lddy, 2));
  if (any_dw) {
    v.reads(view(r.X, r.M, r.K, r.ldx, 2));
    v.reads(view(r.x_codes, 1, r.M * r.K, 0, 1));
    v.reads(view(r.x_scales, 1, r.M * scale_cols(r.K), 0, 1));
  }
  if (any_dx) v.reads(view(r.W, wr, wc, r.ldw, 2));
  if (act) {
    v.reads(view(r.Z, r.M, r.N, r.ldz, 2));
    v.reads(view(r.z_codes, 1, r.M * r.N, 0, 1));
    v.reads(view(r.z_scales, 1, r.M * scale_cols(r.N), 0, 1));
  }
  v.writes(view(r.dX, r.M, r.K, r.lddx, 2));
  v.writes(view(r.dW, wr, wc, r.lddw, elem_bytes(r.dw_dtype)));
  v.writes(view(r.dbias, 1, r.N, 0, elem_bytes(r.bias_dtype)));
  v.writes(view(need ? ws : nullptr, 1, need, 0, 1));
  return v.clash() ? MMAEMU_ERR_ALIAS : MMAEMU_OK;
}

template <int DT>
hipError_t dz_launch(const DzArgs& d, int64_t runs, hipStream_t s) {
  const dim3 grid((uint32_t)((d.N + 511) / 512), (uint32_t)runs);
  dz_kernel<DT><<<grid, 256, 0, s>>>(d);
  return hipGetLastError();
}

// rows of zeros (a gradient over no rows)
__global__ void zero_rows_kernel(void* p, int64_t ld, int64_t rows, int64_t cols, int dt) {
  const int64_t n = rows * cols;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    store_any(p, i / cols * ld + i % cols, 0.0f, dt);
}

}  // namespace

hipError_t mmaops::zero_rows(void* p, int64_t ld, int64_t rows, int64_t cols, int dt,
                             hipStream_t s) {
  if (!p || rows == 0 || cols == 0) return hipSuccess;
  const int64_t blocks = (rows * cols + 255) / 256;
  zero_rows_kernel<<<(uint32_t)(blocks < 4096 ? blocks : 4096), 256, 0, s>>>(p, ld, rows, cols,
                                                                             dt);
  return hipGetLastError();
}

namespace {

hipError_t backward_run(const mma_linear_backward_args& r, void* ws, hipStream_t s) {
  const int64_t wr = r.w_transposed ? r.N : r.K, wc = r.w_transposed ? r.K : r.N;
  if (r.M == 0 || r.N == 0) {  // sums over nothing
    hipError_t e = zero_rows(r.dX, r.lddx, r.M, r.K, r.dtype, s);
    if (e == hipSuccess) e = zero_rows(r.dW, r.lddw, wr, wc, r.dw_dtype, s);
    if (e == hipSuccess) e = zero_rows(r.dbias, r.N, 1, r.N, r.bias_dtype, s);
    return e;
  }
  const BackwardPlan b = backward_plan(r, ws);
  char* const base = (char*)ws;
  hipError_t e = hipSuccess;
  if (b.has_dz || r.dbias) {
    DzArgs d;
    memset(&d, 0, sizeof d);
    d.dy = r.dY;
    d.lddy = r.lddy;
    d.z = r.Z;
    d.ldz = r.ldz;
    d.codes = r.z_codes;
    d.scales = r.z_scales;
    d.dz = b.has_dz ? base + b.dz_at : nullptr;
    d.lddz = (r.N + 7) / 8 * 8;
    d.partial = r.dbias ? (float*)(base + b.db_at) : nullptr;
    d.M = r.M;
    d.N = r.N;
    d.act = r.activation;
    int64_t runs = b.db_runs;
    d.run = b.db_run;
    if (!r.dbias) {
      runs = (r.M + 7) / 8 < 4096 ? (r.M + 7) / 8 : 4096;
      d.run = (r.M + runs - 1) / runs;
    }
    e = r.dtype == kFP16 ? dz_launch<kFP16>(d, runs, s) : dz_launch<kBF16>(d, runs, s);
    if (e != hipSuccess) return e;
    if (r.dbias && !b.pair) {
      e = column_sums(d.partial, b.db_runs, r.N, r.dbias, nullptr, 0, r.bias_dtype, s);
      if (e != hipSuccess) return e;
    }
  }
  if (r.dW && r.K && r.x_codes) {
    e = restore_to(r.dtype, r.x_codes, r.x_scales, base + b.x_at, (r.K + 7) / 8 * 8, r.M, r.K, s);
    if (e != hipSuccess) return e;
  }
  LinearArgs gx, gw;
  memset(&gx, 0, sizeof gx);
  memset(&gw, 0, sizeof gw);
  gx.y = r.dX;
  gx.ldy = r.lddx;
  gx.out_dt = r.dtype;
  gw.y = r.dW;
  gw.ldy = r.lddw;
  gw.out_dt = r.dw_dtype;
  if (b.pair) {
    PairArgs p;
    memset(&p, 0, sizeof p);
    e = linear_fill(b.dx, b.pdx, gx, base + b.part_at, s);
    if (e == hipSuccess) e = linear_fill(b.dw, b.pdw, gw, base + b.part2_at, s);
    if (e != hipSuccess) return e;
    p.dx = gx;
    p.dw = gw;
    p.partial = (const float*)(base + b.db_at);
    p.dbias = r.dbias;
    p.cols = r.N;
    p.count = b.db_runs;
    p.dbias_dt = r.bias_dtype;
    return r.dtype == kFP16 ? pair_launch_fp16(b.dx.lb, p, s) : pair_launch_bf16(b.dx.lb, p, s);
  }
  if (r.dX && r.K) {
    e = linear_run(r.dtype, b.dx, b.pdx, gx, base + b.part_at, s);
    if (e != hipSuccess) return e;
  }
  if (r.dW && r.K) e = linear_run(r.dtype, b.dw, b.pdw, gw, base + b.part2_at, s);
  return e;
}

int64_t norm_backward_need(int64_t rows, int64_t cols) {
  // the larger of the two vector widths' plans, as the type is not given
  const int a = norm_backward_groups(rows, cols, 8), b = norm_backward_groups(rows, cols, 4);
  return up256((int64_t)(a > b ? a : b) * 2 * cols * 4);
}

}  // namespace

extern "C" {

int mma_layer_norm(int dtype, int param_dtype, const void* X, int64_t ldx, const void* weight,
                   const void* bias, void* Y, int64_t ldy, float* mean, float* rstd,
                   uint8_t* codes, uint8_t* scales, int64_t rows, int64_t cols, float eps,
                   void* hip_stream) {
  if (!any_type(dtype) || !param_type_ok(dtype, param_dtype)) return MMAEMU_ERR_DTYPE;
  if (cols < 1 || !shape_ok(rows, cols, ldx) || !shape_ok(rows, cols, ldy))
    return MMAEMU_ERR_SHAPE;
  if (rows == 0) return MMAEMU_OK;
  if (!X || !Y || !mean != !rstd || !codes != !scales) return MMAEMU_ERR_NULL;
  const int e = elem_bytes(dtype), pe = elem_bytes(param_dtype);
  if (!aligned(X, e) || !aligned(Y, e) || !aligned(weight, pe) || !aligned(bias, pe) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return MMAEMU_ERR_ALIGN;
  Views v;
  v.reads(view(X, rows, cols, ldx, e));
  v.reads(view(weight, 1, cols, 0, pe));
  v.reads(view(bias, 1, cols, 0, pe));
  v.writes(view(Y, rows, cols, ldy, e));
  v.writes(view(mean, 1, rows, 0, 4));
  v.writes(view(rstd, 1, rows, 0, 4));
  v.writes(view(codes, 1, rows * cols, 0, 1));
  v.writes(view(scales, 1, rows * scale_cols(cols), 0, 1));
  if (v.clash()) return MMAEMU_ERR_ALIAS;
  NormArgs a;
  memset(&a, 0, sizeof a);
  a.x = X;
  a.ldx = ldx;
  a.weight = weight;
  a.bias = bias;
  a.y = Y;
  a.ldy = ldy;
  a.mean = mean;
  a.rstd = rstd;
  a.codes_out = codes;
  a.scales_out = scales;
  a.rows = rows;
  a.cols = (int)cols;
  a.eps = eps;
  (void)hipGetLastError();
  const hipError_t err =
      MMAOPS_BY_TYPES(dtype, param_dtype, norm_launch, a, (hipStream_t)hip_stream);
  return err == hipSuccess ? MMAEMU_OK : hip_fail(err, "mma_layer_norm launch");
}

int64_t mma_layer_norm_backward_workspace(int64_t rows, int64_t cols) {
  if (cols < 1 || rows < 1 || !shape_ok(rows, cols, cols)) return 0;
  return norm_backward_need(rows, cols);
}

int mma_layer_norm_backward(int dtype, int param_dtype, const void* dY, int64_t lddy,
                            const void* X, int64_t ldx, const uint8_t* codes,
                            const uint8_t* scales, const void* weight, const float* mean,
                            const float* rstd, void* dX, int64_t lddx, void* dweight,
                            void* dbias, int64_t rows, int64_t cols, void* workspace,
                            int64_t workspace_bytes, void* hip_stream) {
  if (!any_type(dtype) || !param_type_ok(dtype, param_dtype)) return MMAEMU_ERR_DTYPE;
  if (cols < 1 || !shape_ok(rows, cols, lddy) || (X && !shape_ok(rows, cols, ldx)) ||
      (dX && !shape_ok(rows, cols, lddx)))
    return MMAEMU_ERR_SHAPE;
  const hipStream_t s = (hipStream_t)hip_stream;
  const int e = elem_bytes(dtype), pe = elem_bytes(param_dtype);
  const bool sums = dweight || dbias;
  if (!sums && (!dX || rows == 0)) return MMAEMU_OK;
  if (!aligned(dweight, pe) || !aligned(dbias, pe)) return MMAEMU_ERR_ALIGN;
  if (rows == 0) {
    if (overlap(view(dweight, 1, cols, 0, pe), view(dbias, 1, cols, 0, pe)))
      return MMAEMU_ERR_ALIAS;
    (void)hipGetLastError();
    hipError_t err = zero_rows(dweight, cols, 1, cols, param_dtype, s);
    if (err == hipSuccess) err = zero_rows(dbias, cols, 1, cols, param_dtype, s);
    return err == hipSuccess ? MMAEMU_OK : hip_fail(err, "mma_layer_norm_backward launch");
  }
  if (!dY || !X == !codes || !codes != !scales || !mean || !rstd) return MMAEMU_ERR_NULL;
  if (!aligned(dY, e) || !aligned(X, e) || !aligned(dX, e) || !aligned(weight, pe) ||
      !aligned(mean, 4) || !aligned(rstd, 4) || (workspace && !aligned(workspace, 256)))
    return MMAEMU_ERR_ALIGN;
  const int64_t need = sums ? norm_backward_need(rows, cols) : 0;
  if (need && (!workspace || workspace_bytes < need)) return MMAEMU_ERR_SCRATCH;
  Views v;
  if (!(dX == dY && lddx == lddy)) v.reads(view(dY, rows, cols, lddy, e));
  v.reads(view(X, rows, cols, ldx, e));
  v.reads(view(codes, 1, rows * cols, 0, 1));
  v.reads(view(scales, 1, rows * scale_cols(cols), 0, 1));
  v.reads(view(weight, 1, cols, 0, pe));
  v.reads(view(mean, 1, rows, 0, 4));
  v.reads(view(rstd, 1, rows, 0, 4));
  v.writes(view(dX, rows, cols, lddx, e));
  v.writes(view(dweight, 1, cols, 0, pe));
  v.writes(view(dbias, 1, cols, 0, pe));
  v.writes(view(need ? workspace : nullptr, 1, need, 0, 1));
  if (v.clash()) return MMAEMU_ERR_ALIAS;
  NormArgs a;
  memset(&a, 0, sizeof a);
  a.x = X;
  a.ldx = ldx;
  a.codes = codes;
  a.scales = scales;
  a.weight = weight;
  a.y = dX;
  a.ldy = lddx;
  a.mean = (float*)mean;
  a.rstd = (float*)rstd;
  a.rows = rows;
  a.cols = (int)cols;
  a.dy = dY;
  a.lddy = lddy;
  a.partial = sums ? (float*)workspace : nullptr;
  const int groups = norm_backward_groups(rows, cols, dtype == kFP32 ? 4 : 8);
  (void)hipGetLastError();
  hipError_t err = MMAOPS_BY_TYPES(dtype, param_dtype, norm_backward_launch, a, groups, s);
  if (err == hipSuccess && sums)
    err = column_sums(a.partial, groups, cols, dweight, dbias, 1, param_dtype, s);
  return err == hipSuccess ? MMAEMU_OK : hip_fail(err, "mma_layer_norm_backward launch");
}

int mma_checkpoint(int dtype, const void* X, int64_t ldx, uint8_t* codes, uint8_t* scales,
                   int64_t rows, int64_t cols, void* hip_stream) {
  if (!any_type(dtype)) return MMAEMU_ERR_DTYPE;
  if (!shape_ok(rows, cols, ldx)) return MMAEMU_ERR_SHAPE;
  if (rows == 0 || cols == 0) return MMAEMU_OK;
  if (!X || !codes || !scales) return MMAEMU_ERR_NULL;
  if (!aligned(X, elem_bytes(dtype))) return MMAEMU_ERR_ALIGN;
  Views v;
  v.reads(view(X, rows, cols, ldx, elem_bytes(dtype)));
  v.writes(view(codes, 1, rows * cols, 0, 1));
  v.writes(view(scales, 1, rows * scale_cols(cols), 0, 1));
  if (v.clash()) return MMAEMU_ERR_ALIAS;
  const hipStream_t s = (hipStream_t)hip_stream;
  (void)hipGetLastError();
  const hipError_t err =
      dtype == kFP16   ? save_launch<kFP16>(X, ldx, codes, scales, rows, cols, s)
      : dtype == kBF16 ? save_launch<kBF16>(X, ldx, codes, scales, rows, cols, s)
                       : save_launch<kFP32>(X, ldx, codes, scales, rows, cols, s);
  return err == hipSuccess ? MMAEMU_OK : hip_fail(err, "mma_checkpoint launch");
}

int mma_restore(int dtype, const uint8_t* codes, const uint8_t* scales, void* Y, int64_t ldy,
                int64_t rows, int64_t cols, void* hip_stream) {
  if (!any_type(dtype)) return MMAEMU_ERR_DTYPE;
  if (!shape_ok(rows, cols, ldy)) return MMAEMU_ERR_SHAPE;
  if (rows == 0 || cols == 0) return MMAEMU_OK;
  if (!Y || !codes || !scales) return MMAEMU_ERR_NULL;
  if (!aligned(Y, elem_bytes(dtype))) return MMAEMU_ERR_ALIGN;
  Views v;
  v.reads(view(codes, 1, rows * cols, 0, 1));
  v.reads(view(scales, 1, rows * scale_cols(cols), 0, 1));
  v.writes(view(Y, rows, cols, ldy, elem_bytes(dtype)));
  if (v.clash()) return MMAEMU_ERR_ALIAS;
  (void)hipGetLastError();
  const hipError_t err =
      restore_to(dtype, codes, scales, Y, ldy, rows, cols, (hipStream_t)hip_stream);
  return err == hipSuccess ? MMAEMU_OK : hip_fail(err, "mma_restore launch");
}

int64_t mma_linear_workspace(const mma_linear_args* args) {
  if (!args || check_linear(*args, 0, nullptr, true) != MMAEMU_OK) return 0;
  return linear_need(*args);
}

int mma_linear(const mma_linear_args* args, void* workspace, int64_t workspace_bytes,
               void* hip_stream) {
  if (!args) return MMAEMU_ERR_NULL;
  const mma_linear_args& r = *args;
  const int rc = check_linear(r, workspace_bytes, workspace, false);
  if (rc || r.M == 0 || r.N == 0) return rc;
  LinearArgs g;
  memset(&g, 0, sizeof g);
  g.bias = r.bias;
  g.residual = r.residual;
  g.y = r.Y;
  g.z = r.Z;
  g.codes = r.codes;
  g.scales = r.scales;
  g.ldr = r.ldr;
  g.ldy = r.ldy;
  g.ldz = r.ldz;
  g.bias_dt = r.bias_dtype;
  g.out_dt = r.out_dtype;
  g.act = r.activation;
  const Product p = forward_product(r);
  (void)hipGetLastError();
  const hipError_t err = linear_run(r.dtype, p, linear_plan(p, r.codes != nullptr), g, workspace,
                                    (hipStream_t)hip_stream);
  return err == hipSuccess ? MMAEMU_OK : hip_fail(err, "mma_linear launch");
}

int64_t mma_linear_backward_workspace(const mma_linear_backward_args* args) {
  if (!args || check_backward(*args, 0, nullptr, true) != MMAEMU_OK) return 0;
  if (args->M == 0 || args->N == 0) return 0;
  return backward_plan(*args, nullptr).bytes;
}

int mma_linear_backward(const mma_linear_backward_args* args, void* workspace,
                        int64_t workspace_bytes, void* hip_stream) {
  if (!args) return MMAEMU_ERR_NULL;
  const int rc = check_backward(*args, workspace_bytes, workspace, false);
  if (rc) return rc;
  (void)hipGetLastError();
  const hipError_t err = backward_run(*args, workspace, (hipStream_t)hip_stream);
  return err == hipSuccess ? MMAEMU_OK : hip_fail(err, "mma_linear_backward launch");
}

const char* mma_ops_strerror(int code) {
  switch (code) {
    case MMAEMU_OK: return "ok";
    case MMAEMU_ERR_DTYPE:
      return "unsupported element type (products take FP16 and BF16; a parameter or output "
             "type is the operands' or FP32)";
    case MMAEMU_ERR_UNSUPPORTED: 
      return "unknown activation or norm, a flag other than 0 or 1, or a probability outside "
             "[0, 1]";
    case MMAEMU_ERR_SHAPE:
      return "bad shape (negative or too large, a leading dimension below the row length, or "
             "a layer norm over no columns)";
    case MMAEMU_ERR_NULL:
      return "a required pointer is NULL (codes and scales, mean and rstd come in pairs; a "
             "matrix or its checkpoint, not both)";
    case MMAEMU_ERR_ALIAS: return "an output overlaps an input or another output";
    case MMAEMU_ERR_ALIGN:
      return "a pointer is not aligned to its elements (the workspace: to 256 bytes)";
    case MMAEMU_ERR_SCRATCH: return "the workspace is missing or smaller than the call needs";
    case MMAEMU_ERR_HIP: return g_hip_error;
    default: return "unknown error code";
  }
}

}  // extern "C"
