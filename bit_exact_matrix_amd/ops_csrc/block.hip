// block.hip -- the C ABI of the gated block's operators (include/mmaops.h):
// argument checks and launches.
#include <math.h>
#include <string.h>

#include "../../include/mmaops.h"
#include "checks.h"
#include "gated.h"
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
  DropGrid cut{4, 0, 0};
  while (cut.shift < 8 && (int64_t(1) << cut.shift) < vecs) ++cut.shift;
  const bool exact = vecs <= 128 && vecs != (int64_t(1) << cut.shift);
  cut.lanes = exact ? (int)vecs : 1 << cut.shift;
  cut.inverse = 65536 / cut.lanes + 1;
  const int64_t per = 256 / cut.lanes, gx = (rows + per - 1) / per;
  const int64_t gy = (vecs + cut.lanes - 1) / cut.lanes;
  const dim3 grid((uint32_t)(gx < (1 << 22) ? gx : (1 << 22)), (uint32_t)(gy < 256 ? gy : 256));
  if (exact)
    dropout_kernel<DT, true><<<grid, 256, 0, s>>>(x, ldx, residual, ldr, y, ldy, rows, cols, d,
                                                  cut);
  else
    dropout_kernel<DT, false><<<grid, 256, 0, s>>>(x, ldx, residual, ldr, y, ldy, rows, cols, d,
                                                   cut);
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

// The arguments without those that the call does not read: the vectors of a norm
// that is not there, whose pointers may be anything, and what goes with them.  The
// checks and the kernels see only what is left.
mma_residual_norm_args in_use(mma_residual_norm_args r) {
  if (r.post == kNormNone) {
    r.post_weight = r.post_bias = nullptr;
    r.post_mean = r.post_rstd = nullptr;
  }
  if (r.pre == kNormNone) {
    r.pre_weight = r.pre_bias = nullptr;
    r.mean = r.rstd = nullptr;
    r.H = nullptr;
  }
  return r;
}

mma_residual_norm_backward_args in_use(mma_residual_norm_backward_args r) {
  if (r.post == kNormNone) {
    r.post_weight = r.post_bias = nullptr;
    r.post_rstd = nullptr;
    if (!r.dgate) r.branch = nullptr;
  }
  if (r.pre == kNormNone) {
    r.dH = r.R = r.pre_weight = nullptr;
    r.rstd = nullptr;
  }
  if (r.post != kNormLayer) r.post_mean = nullptr;
  if (r.pre != kNormLayer) r.mean = nullptr;
  return r;
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

// How a row is held: waves a row and vectors a lane; no waves where it is too
// long for registers.
struct RowPlan {
  int waves, nv;
};

// One vector a lane and as many waves as the row needs, up to 16; then two.
RowPlan row_plan(int64_t cols, int V) {
  const int64_t vecs = (cols + V - 1) / V;
  if (vecs <= 1024) return {(int)((vecs + 63) / 64), 1};
  if (vecs > 2048) return {0, 0};
  return {(int)((vecs + 127) / 128), 2};
}

// Workgroups of a row's waves (four rows of one wave), as many as the CUs
// hold at once: 20 waves with one vector a lane, 16 with two.
template <int DT, int PDT, int W, int NV>
void join_run(const JoinArgs& a, int waves, hipStream_t s) {
  constexpr int G = W == 1 ? 4 : 1;
  const int64_t groups = (a.rows + G - 1) / G, per = (NV == 1 ? 20 : 16) / (waves * G);
  const int64_t most = kCUs * (per > 1 ? per : 1);
  join_kernel<DT, PDT, W, NV, G>
      <<<(uint32_t)(groups < most ? groups : most), waves * 64 * G, 0, s>>>(a);
}

template <int DT, int PDT>
hipError_t join_launch(const JoinArgs& a, hipStream_t s) {
  const RowPlan p = row_plan(a.cols, kVec<DT>);
  if (p.waves == 0) {
    const uint32_t grid = (uint32_t)(a.rows < 2 * kCUs ? a.rows : 2 * kCUs);
    join_long_kernel<DT, PDT><<<grid, 1024, 0, s>>>(a);
  } else if (p.nv == 2) {
    join_run<DT, PDT, 16, 2>(a, p.waves, s);
  } else if (p.waves == 1) {
    join_run<DT, PDT, 1, 1>(a, 1, s);
  } else if (p.waves <= 4) {
    join_run<DT, PDT, 4, 1>(a, p.waves, s);
  } else if (p.waves <= 8) {
    join_run<DT, PDT, 8, 1>(a, p.waves, s);
  } else {
    join_run<DT, PDT, 16, 1>(a, p.waves, s);
  }
  return hipGetLastError();
}

// The backward pass: elements a lane and waves a row (8 elements of FP32, two
// vectors, take the registers that one vector of the 16-bit types does: 3276 x 5120
// 212 us in several passes over the rows, in one 127, with biases 186), and the rows
// that a workgroup works on at a time.
struct BackPlan {
  int v, waves, rows;  // waves 0: in several passes
};
BackPlan back_plan(int64_t cols, int dt) {
  const int one = dt == kFP32 ? 4 : 8;
  for (int v = one; v <= 8; v *= 2) {
    const int64_t waves = (cols + 64 * v - 1) / (64 * v);
    if (waves <= 16) {
      const int w = (int)waves;
      return {v, w, w <= 2 ? 8 / w : w <= 4 ? 2 : 1};
    }
  }
  return {one, 0, 32};
}

// The launch and its workspace: the groups' column sums, then the rows' means
// where a row is read in several passes, or what the kernel asks for spare rows.
struct JoinPlan {
  int groups;        // workgroups, or runs of rows of the column pass
  bool sums, shift;  // column sums, those of biases among them
  int64_t means_at;  // the rows' means, or the spare rows
  int64_t bytes;
};

// Workgroups as many as the CUs hold at once, 16 waves each, with a row of
// partial sums for each.
JoinPlan join_plan(const mma_residual_norm_backward_args& r) {
  JoinPlan p{};
  if (r.rows == 0) return p;
  p.sums = r.dgate || r.dpost_weight || r.dpost_bias || r.dpre_weight || r.dpre_bias;
  p.shift = r.dpre_bias || r.dpost_bias || (r.dgate && r.post != kNormNone && r.post_bias);
  const BackPlan b = back_plan(r.cols, r.dtype);
  const int waves = b.waves;
  const int64_t per = b.rows, runs = (r.rows + per - 1) / per;
  const int64_t most = kCUs * (waves && waves <= 8 ? 16 / (waves * per) : 1);
  p.groups = (int)(runs < most ? runs : most);
  if (!p.sums) return p;
  p.means_at = up256((int64_t)p.groups * 4 * r.cols * 4);
  const int64_t spare =
      waves && !r.dX && !r.dbranch ? p.groups * per * r.cols * elem_bytes(r.dtype) : 0;
  p.bytes = p.means_at + up256(waves ? spare : r.rows * 8);
  return p;
}

int check_join_backward(const mma_residual_norm_backward_args& r, int64_t ws_bytes,
                        const void* ws, bool sizes_only, DropArgs* d) {
  const int rc = join_head(r, d);
  if (rc) return rc;
  if (r.reserved) return MMAEMU_ERR_UNSUPPORTED;
  const bool post = r.post != kNormNone, pre = r.pre != kNormNone;
  if (r.cols < 1 || (r.dR && !shape_ok(r.rows, r.cols, r.lddr)) ||
      (pre && (!shape_ok(r.rows, r.cols, r.lddh) || !shape_ok(r.rows, r.cols, r.ldr))) ||
      (r.branch && !shape_ok(r.rows, r.cols, r.ldb)) ||
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
  v.reads(view(r.dH, r.rows, r.cols, r.lddh, e));
  v.reads(view(r.R, r.rows, r.cols, r.ldr, e));
  v.reads(view(r.branch, r.rows, r.cols, r.ldb, e));
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

template <int DT, int PDT, int V, int W, int G, bool SHIFT>
hipError_t join_backward_run(const JoinArgs& a, int waves, int groups, hipStream_t s) {
  if (a.cols == waves * 64 * V)
    join_backward_kernel<DT, PDT, V, W, G, SHIFT, true>
        <<<(uint32_t)groups, waves * 64 * G, 0, s>>>(a);
  else
    join_backward_kernel<DT, PDT, V, W, G, SHIFT, false>
        <<<(uint32_t)groups, waves * 64 * G, 0, s>>>(a);
  return hipGetLastError();
}

template <int DT, int PDT, int V, int W, int G>
hipError_t join_backward_run(const JoinArgs& a, int waves, int groups, bool shift, hipStream_t s) {
  return shift ? join_backward_run<DT, PDT, V, W, G, true>(a, waves, groups, s)
               : join_backward_run<DT, PDT, V, W, G, false>(a, waves, groups, s);
}

template <int DT, int PDT>
hipError_t join_backward_launch(const JoinArgs& a, int groups, bool shift, hipStream_t s) {
  constexpr int V = kVec<DT>;
  const BackPlan b = back_plan(a.cols, DT);
  if constexpr (DT == kFP32) {
    if (b.v == 8) return join_backward_run<DT, PDT, 8, 16, 1>(a, b.waves, groups, shift, s);
  }
  switch (b.waves) {  // the rows at a time: back_plan
    case 0: break;
    case 1: return join_backward_run<DT, PDT, V, 1, 8>(a, 1, groups, shift, s);
    case 2: return join_backward_run<DT, PDT, V, 2, 4>(a, 2, groups, shift, s);
    case 3: return join_backward_run<DT, PDT, V, 3, 2>(a, 3, groups, shift, s);
    case 4: return join_backward_run<DT, PDT, V, 4, 2>(a, 4, groups, shift, s);
    default:
      return b.waves <= 8 ? join_backward_run<DT, PDT, V, 8, 1>(a, b.waves, groups, shift, s)
                          : join_backward_run<DT, PDT, V, 16, 1>(a, b.waves, groups, shift, s);
  }
  const uint32_t grid = (uint32_t)(a.rows < 2 * kCUs ? a.rows : 2 * kCUs);
  join_long_dx_kernel<DT, PDT><<<grid, 1024, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.partial) return e;
  const dim3 sums((uint32_t)((a.cols + 64 * V - 1) / (64 * V)), (uint32_t)groups);
  join_long_sums_kernel<DT, PDT><<<sums, 256, 0, s>>>(a, (a.rows + groups - 1) / groups);
  return hipGetLastError();
}

// -------------------------------------------------------- gated layer
GatedLaunches launches(int dt) { return dt == kFP16 ? gated_fp16() : gated_bf16(); }

// Two matrices of 16-bit elements copied to rows that start on 16 bytes, in
// one launch (as align_kernel).
__global__ __launch_bounds__(256) void align_two_kernel(const uint16_t* x, int64_t ldx,
                                                        uint16_t* y, const uint16_t* x2,
                                                        int64_t ldx2, uint16_t* y2, int64_t ldy,
                                                        int64_t rows, int64_t cols) {
  constexpr int V = 8, kLanes = 64;
  const bool two = blockIdx.z != 0;
  const uint16_t* const from = two ? x2 : x;
  const int64_t ld = two ? ldx2 : ldx;
  uint16_t* const to = two ? y2 : y;
  const int lane = threadIdx.x % kLanes, g = threadIdx.x / kLanes;
  const int64_t step = (int64_t)gridDim.x * (256 / kLanes);
  const int64_t cstep = (int64_t)gridDim.y * kLanes * V;
  for (int64_t row = (int64_t)blockIdx.x * (256 / kLanes) + g; row < rows; row += step)
    for (int64_t c = ((int64_t)blockIdx.y * kLanes + lane) * V; c < cols; c += cstep) {
      const int n = cols - c < V ? (int)(cols - c) : V;
      store_pack<kBF16, V>((__bf16*)(to + row * ldy + c),
                           load_pack<kBF16, V>((const __bf16*)(from + row * ld + c), n), V);
    }
}

hipError_t align_two(const void* x, int64_t ldx, void* y, const void* x2, int64_t ldx2, void* y2,
                     const Stored& t, hipStream_t s) {
  if (t.rows == 0 || t.cols == 0) return hipSuccess;
  const int64_t gx = (t.rows + 3) / 4, gy = (t.cols + 511) / 512;
  const dim3 grid((uint32_t)(gx < (1 << 22) ? gx : (1 << 22)), (uint32_t)(gy < 256 ? gy : 256), 2);
  align_two_kernel<<<grid, 256, 0, s>>>((const uint16_t*)x, ldx, (uint16_t*)y,
                                        (const uint16_t*)x2, ldx2, (uint16_t*)y2, t.ld, t.rows,
                                        t.cols);
  return hipGetLastError();
}

// A pair's arguments, with its operands copied where the plan says so.
hipError_t paired_fill(const Paired& q, const Plan& r, LinearArgs& g, const void*& a2,
                       const void*& b2, void* ws, hipStream_t s) {
  const Product& p = q.p;
  const TileShape& t = kTileShape[r.tile];
  const int cols = paired_columns(q.kind, r.tile);
  g.a = p.a;
  g.b = p.b;
  g.lda = p.lda;
  g.ldb = p.ldb;
  a2 = q.a2 ? q.a2 : p.a;
  b2 = q.b2 ? q.b2 : p.b;
  char* at = (char*)ws + paired_partial_bytes(q, r);
  auto copy = [&](const void*& one, const void*& two, bool second, int64_t ld2, int64_t& ld,
                  const Stored& st) {
    char* const to = at;
    at += copy_bytes(true, st) * (second ? 2 : 1);
    char* const to2 = second ? to + copy_bytes(true, st) : to;
    const hipError_t e = second ? align_two(one, ld, to, two, ld2, to2, st, s)
                                : align_rows(one, ld, to, st, s);
    one = to;
    two = to2;
    ld = st.ld;
    return e;
  };
  if (r.copy_a) {
    const hipError_t e =
        copy(g.a, a2, q.a2 != nullptr, q.lda2, g.lda, stored(p.la, p.M, p.K));
    if (e != hipSuccess) return e;
  }
  if (r.copy_b) {
    const hipError_t e =
        copy(g.b, b2, q.b2 != nullptr, q.ldb2, g.ldb, stored(p.lb, p.N, p.K));
    if (e != hipSuccess) return e;
  }
  g.M = p.M;
  g.N = p.N;
  g.K = p.K;
  g.splits = r.splits;
  g.guard = r.guard;
  g.tiles_m = (int)((p.M + t.bm - 1) / t.bm);
  g.tiles_n = (int)((p.N + cols - 1) / cols);
  g.partial = r.partial ? (float*)ws : nullptr;
  return hipSuccess;
}

// sizes whose products and tile counts the 64-bit and 31-bit counters hold
bool gated_shape_ok(int64_t M, int64_t N, int64_t K) {
  constexpr int64_t kMax = kMaxCols;
  if (M < 0 || N < 0 || K < 0 || M > kMax || N > kMax || K > kMax) return false;
  return ((M + 15) / 16) * ((N + 15) / 16) <= INT32_MAX / 2 &&
         ((M + 15) / 16) * ((K + 15) / 16) <= INT32_MAX / 2 &&
         ((N + 15) / 16) * ((K + 15) / 16) <= INT32_MAX / 2;
}

Paired gated_product(const mma_gated_linear_args& r) {
  return Paired{kGated,
                Product{r.M, r.N, r.K, 0, r.w_transposed ? 0 : 1, r.X, r.Wg, r.ldx, r.ldwg},
                nullptr, r.Wu, 0, r.ldwu};
}

int64_t gated_need(const mma_gated_linear_args& r) {
  if (r.M == 0 || r.N == 0) return 0;
  const Paired q = gated_product(r);
  return paired_bytes(q, paired_plan(q, r.g_codes != nullptr));
}

template <typename ARGS>
int gated_head(const ARGS& r, int out_dtype) {
  if (!half_type(r.dtype)) return MMAEMU_ERR_DTYPE;
  if (!param_type_ok(r.dtype, out_dtype) || !param_type_ok(r.dtype, r.bias_dtype))
    return MMAEMU_ERR_DTYPE;
  if (r.activation < MMAOPS_ACT_NONE || r.activation > MMAOPS_ACT_SILU || r.reserved ||
      (r.w_transposed & ~1))
    return MMAEMU_ERR_UNSUPPORTED;
  return gated_shape_ok(r.M, r.N, r.K) ? MMAEMU_OK : MMAEMU_ERR_SHAPE;
}

int check_gated(const mma_gated_linear_args& r, int64_t ws_bytes, const void* ws,
                bool sizes_only) {
  const int rc = gated_head(r, r.out_dtype);
  if (rc || sizes_only) return rc;
  const int64_t wr = r.w_transposed ? r.N : r.K, wc = r.w_transposed ? r.K : r.N;
  if (!shape_ok(r.M, r.K, r.ldx) || !shape_ok(wr, wc, r.ldwg) || !shape_ok(wr, wc, r.ldwu) ||
      !shape_ok(r.M, r.N, r.ldy) || (r.G && !shape_ok(r.M, r.N, r.ldg)) ||
      (r.U && !shape_ok(r.M, r.N, r.ldu)))
    return MMAEMU_ERR_SHAPE;
  if (r.M == 0 || r.N == 0) return MMAEMU_OK;
  if (!r.Y || (r.K && (!r.X || !r.Wg || !r.Wu)) || !r.G != !r.U || !r.g_codes != !r.g_scales ||
      !r.g_codes != !r.u_codes || !r.g_codes != !r.u_scales)
    return MMAEMU_ERR_NULL;
  const int oe = elem_bytes(r.out_dtype), be = elem_bytes(r.bias_dtype);
  if (!aligned(r.X, 2) || !aligned(r.Wg, 2) || !aligned(r.Wu, 2) || !aligned(r.Y, oe) ||
      !aligned(r.G, 2) || !aligned(r.U, 2) || !aligned(r.bias_g, be) || !aligned(r.bias_u, be) ||
      (ws && !aligned(ws, 256)))
    return MMAEMU_ERR_ALIGN;
  const int64_t need = gated_need(r);
  if (need && (!ws || ws_bytes < need)) return MMAEMU_ERR_SCRATCH;
  Views v;
  if (r.K) {
    v.reads(view(r.X, r.M, r.K, r.ldx, 2));
    v.reads(view(r.Wg, wr, wc, r.ldwg, 2));
    v.reads(view(r.Wu, wr, wc, r.ldwu, 2));
  }
  v.reads(view(r.bias_g, 1, r.N, 0, be));
  v.reads(view(r.bias_u, 1, r.N, 0, be));
  v.writes(view(r.Y, r.M, r.N, r.ldy, oe));
  v.writes(view(r.G, r.M, r.N, r.ldg, 2));
  v.writes(view(r.U, r.M, r.N, r.ldu, 2));
  for (const uint8_t* codes : {r.g_codes, r.u_codes}) v.writes(view(codes, 1, r.M * r.N, 0, 1));
  for (const uint8_t* scales : {r.g_scales, r.u_scales})
    v.writes(view(scales, 1, r.M * scale_cols(r.N), 0, 1));
  v.writes(view(need ? ws : nullptr, 1, need, 0, 1));
  return v.clash() ? MMAEMU_ERR_ALIAS : MMAEMU_OK;
}

// The backward pass: what it needs of the workspace, piece by piece.
struct GatedBackward {
  Paired dx, dw;
  Plan pdx, pdw;
  bool has_dz;     // dg and du are written
  int db_runs;     // rows of column sums, 0: no bias gradient
  int64_t db_run;  // rows of one of them
  int64_t dg_at, du_at, ldd, x_at, db_at, part_at, part2_at, bytes;
  bool small;      // the products and the column sums in one launch
};

GatedBackward gated_backward(const mma_gated_linear_backward_args& r, void* ws) {
  GatedBackward b;
  memset(&b, 0, sizeof b);
  char* const base = (char*)ws;
  int64_t at = 0;
  b.has_dz = r.dX || r.dWg;
  b.ldd = (r.N + 7) / 8 * 8;  // rows that start on 16 bytes: direct loads
  if (b.has_dz) {
    b.dg_at = at;
    at += up256(r.M * b.ldd * 2);
    b.du_at = at;
    at += up256(r.M * b.ldd * 2);
  }
  if (r.x_codes && r.dWg) {
    b.x_at = at;
    at += up256(r.M * ((r.K + 7) / 8 * 8) * 2);
  }
  if (r.dbias_g || r.dbias_u) {
    const int64_t cols = (r.N + 511) / 512;
    int64_t runs = (8 * kCUs + cols - 1) / cols;
    if (runs > (r.M + 3) / 4) runs = (r.M + 3) / 4;  // a row for each wave
    b.db_run = (r.M + runs - 1) / runs;
    b.db_runs = (int)((r.M + b.db_run - 1) / b.db_run);
    b.db_at = at;
    at += up256((int64_t)b.db_runs * 2 * r.N * 4);
  }
  const void *const dg = base + b.dg_at, *const du = base + b.du_at;
  const void* const x = r.x_codes ? base + b.x_at : r.X;
  const int64_t ldx = r.x_codes ? (r.K + 7) / 8 * 8 : r.ldx;
  b.part_at = at;
  int64_t part = 0;
  if (r.dX) {
    b.dx = Paired{kSummed,
                  Product{r.M, r.K, r.N, 0, r.w_transposed ? 1 : 0, dg, r.Wg, b.ldd, r.ldwg}, du,
                  r.Wu, b.ldd, r.ldwu};
    b.pdx = paired_plan(b.dx, false);
    part = paired_bytes(b.dx, b.pdx);
  }
  if (r.dWg) {
    b.dw = r.w_transposed
               ? Paired{kApart, Product{r.N, r.K, r.M, 1, 1, dg, x, b.ldd, ldx}, du, nullptr,
                        b.ldd, 0}
               : Paired{kApart, Product{r.K, r.N, r.M, 1, 1, x, dg, ldx, b.ldd}, nullptr, du, 0,
                        b.ldd};
    b.pdw = paired_plan(b.dw, false);
    const int64_t w = paired_bytes(b.dw, b.pdw);
    part = part > w ? part : w;
  }
  // All on small tiles, whole, and few enough that one grid holds them: one
  // launch.  Their copies, if any, then stand in the workspace side by side.
  auto tiles = [](const Product& p) { return ((p.M + 63) / 64) * ((p.N + 63) / 64); };
  b.small = r.dX && r.dWg && r.K && b.pdx.tile == kTileSmall && b.pdw.tile == kTileSmall &&
            !b.pdx.partial && !b.pdw.partial && tiles(b.dx.p) + 2 * tiles(b.dw.p) <= (1 << 20);
  b.part2_at = b.small ? at + paired_bytes(b.dx, b.pdx) : at;
  b.bytes = b.small ? b.part2_at + paired_bytes(b.dw, b.pdw) : at + part;
  return b;
}

int check_gated_backward(const mma_gated_linear_backward_args& r, int64_t ws_bytes, void* ws,
                         bool sizes_only) {
  const int rc = gated_head(r, r.dw_dtype);
  if (rc || sizes_only) return rc;
  const int64_t wr = r.w_transposed ? r.N : r.K, wc = r.w_transposed ? r.K : r.N;
  if (!shape_ok(r.M, r.N, r.lddy) || (r.X && !shape_ok(r.M, r.K, r.ldx)) ||
      (r.dX && (!shape_ok(wr, wc, r.ldwg) || !shape_ok(wr, wc, r.ldwu))) ||
      (r.G && !shape_ok(r.M, r.N, r.ldg)) || (r.U && !shape_ok(r.M, r.N, r.ldu)) ||
      (r.dX && !shape_ok(r.M, r.K, r.lddx)) || (r.dWg && !shape_ok(wr, wc, r.lddwg)) ||
      (r.dWu && !shape_ok(wr, wc, r.lddwu)))
    return MMAEMU_ERR_SHAPE;
  if (!r.dWg != !r.dWu) return MMAEMU_ERR_NULL;
  const bool any_dx = r.dX && r.M && r.K, any_dw = r.dWg && r.K && r.N;
  const bool any_db = (r.dbias_g || r.dbias_u) && r.N;
  if (!any_dx && !any_dw && !any_db) return MMAEMU_OK;
  if (r.M && r.N) {
    if (!r.dY || (any_dx && (!r.Wg || !r.Wu))) return MMAEMU_ERR_NULL;
    if (!r.x_codes != !r.x_scales || (any_dw && !r.X == !r.x_codes)) return MMAEMU_ERR_NULL;
    if (!r.g_codes != !r.g_scales || !r.g_codes != !r.u_codes || !r.g_codes != !r.u_scales ||
        !r.G != !r.U || !r.G == !r.g_codes)
      return MMAEMU_ERR_NULL;
  }
  const int we = elem_bytes(r.dw_dtype), be = elem_bytes(r.bias_dtype);
  if (!aligned(r.dY, 2) || !aligned(r.X, 2) || !aligned(r.Wg, 2) || !aligned(r.Wu, 2) ||
      !aligned(r.G, 2) || !aligned(r.U, 2) || !aligned(r.dX, 2) || !aligned(r.dWg, we) ||
      !aligned(r.dWu, we) || !aligned(r.dbias_g, be) || !aligned(r.dbias_u, be) ||
      (ws && !aligned(ws, 256)))
    return MMAEMU_ERR_ALIGN;
  const int64_t need = r.M && r.N ? gated_backward(r, ws).bytes : 0;
  if (need && (!ws || ws_bytes < need)) return MMAEMU_ERR_SCRATCH;
  Views v;
  v.reads(view(r.dY, r.M, r.N, r.lddy, 2));
  if (any_dw) {
    v.reads(view(r.X, r.M, r.K, r.ldx, 2));
    v.reads(view(r.x_codes, 1, r.M * r.K, 0, 1));
    v.reads(view(r.x_scales, 1, r.M * scale_cols(r.K), 0, 1));
  }
  if (any_dx) {
    v.reads(view(r.Wg, wr, wc, r.ldwg, 2));
    v.reads(view(r.Wu, wr, wc, r.ldwu, 2));
  }
  v.reads(view(r.G, r.M, r.N, r.ldg, 2));
  v.reads(view(r.U, r.M, r.N, r.ldu, 2));
  for (const uint8_t* codes : {r.g_codes, r.u_codes}) v.reads(view(codes, 1, r.M * r.N, 0, 1));
  for (const uint8_t* scales : {r.g_scales, r.u_scales})
    v.reads(view(scales, 1, r.M * scale_cols(r.N), 0, 1));
  v.writes(view(r.dX, r.M, r.K, r.lddx, 2));
  v.writes(view(r.dWg, wr, wc, r.lddwg, we));
  v.writes(view(r.dWu, wr, wc, r.lddwu, we));
  v.writes(view(r.dbias_g, 1, r.N, 0, be));
  v.writes(view(r.dbias_u, 1, r.N, 0, be));
  v.writes(view(need ? ws : nullptr, 1, need, 0, 1));
  return v.clash() ? MMAEMU_ERR_ALIAS : MMAEMU_OK;
}

hipError_t gated_backward_run(const mma_gated_linear_backward_args& r, void* ws, hipStream_t s) {
  const int64_t wr = r.w_transposed ? r.N : r.K, wc = r.w_transposed ? r.K : r.N;
  hipError_t e = hipSuccess;
  if (r.M == 0 || r.N == 0) {  // sums over nothing
    e = zero_rows(r.dX, r.lddx, r.M, r.K, r.dtype, s);
    if (e == hipSuccess) e = zero_rows(r.dWg, r.lddwg, wr, wc, r.dw_dtype, s);
    if (e == hipSuccess) e = zero_rows(r.dWu, r.lddwu, wr, wc, r.dw_dtype, s);
    if (e == hipSuccess) e = zero_rows(r.dbias_g, r.N, 1, r.N, r.bias_dtype, s);
    if (e == hipSuccess) e = zero_rows(r.dbias_u, r.N, 1, r.N, r.bias_dtype, s);
    return e;
  }
  const GatedLaunches run = launches(r.dtype);
  const GatedBackward b = gated_backward(r, ws);
  char* const base = (char*)ws;
  GateDzArgs d;
  memset(&d, 0, sizeof d);
  d.dy = r.dY;
  d.lddy = r.lddy;
  d.g = r.G;
  d.u = r.U;
  d.ldg = r.ldg;
  d.ldu = r.ldu;
  d.g_codes = r.g_codes;
  d.g_scales = r.g_scales;
  d.u_codes = r.u_codes;
  d.u_scales = r.u_scales;
  d.dg = b.has_dz ? base + b.dg_at : nullptr;
  d.du = b.has_dz ? base + b.du_at : nullptr;
  d.ldd = b.ldd;
  d.partial = b.db_runs ? (float*)(base + b.db_at) : nullptr;
  d.M = r.M;
  d.N = r.N;
  d.act = r.activation;
  d.run = b.db_run;
  int64_t runs = b.db_runs;
  if (!runs) {
    runs = (r.M + 3) / 4 < 4096 ? (r.M + 3) / 4 : 4096;
    d.run = (r.M + runs - 1) / runs;
  }
  e = run.dz(d, runs, s);
  if (e == hipSuccess && b.db_runs && !b.small)
    e = column_sums(d.partial, b.db_runs, r.N, r.dbias_g, r.dbias_u, 1, r.bias_dtype, s);
  if (e == hipSuccess && r.dWg && r.K && r.x_codes)
    e = restore_to(r.dtype, r.x_codes, r.x_scales, base + b.x_at, (r.K + 7) / 8 * 8, r.M, r.K, s);
  SmallArgs all;
  memset(&all, 0, sizeof all);
  if (e == hipSuccess && r.dX && r.K) {
    LongArgs& g = all.dx;
    g.y = r.dX;
    g.ldy = r.lddx;
    g.out_dt = r.dtype;
    e = paired_fill(b.dx, b.pdx, g, g.a2, g.b2, base + b.part_at, s);
    if (e == hipSuccess && !b.small) e = run.both(b.pdx.tile, b.pdx.direct, b.dx.p.lb, g, s);
  }
  if (e == hipSuccess && r.dWg && r.K) {
    TwoArgs& p = all.dw;
    const void *a2, *b2;
    p.one.y = r.dWg;
    p.one.ldy = r.lddwg;
    p.one.out_dt = r.dw_dtype;
    e = paired_fill(b.dw, b.pdw, p.one, a2, b2, base + b.part2_at, s);
    p.two = p.one;
    p.two.a = a2;
    p.two.b = b2;
    p.two.y = r.dWu;
    p.two.ldy = r.lddwu;
    if (p.one.partial) p.two.partial += b.dw.p.M * b.dw.p.N * b.pdw.splits;
    if (e == hipSuccess && !b.small) e = run.two(b.pdw.tile, b.pdw.direct, p, s);
  }
  if (e == hipSuccess && b.small) {
    all.partial = d.partial;
    all.dbias_g = r.dbias_g;
    all.dbias_u = r.dbias_u;
    all.cols = r.N;
    all.count = b.db_runs;
    all.dbias_dt = r.bias_dtype;
    e = run.small(b.dx.p.lb, all, s);
  }
  return e;
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
  const mma_residual_norm_args r = in_use(*args);
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
  a.post_rstd = r.post_rstd;
  a.mean = r.pre == kNormLayer ? r.mean : nullptr;
  a.rstd = r.rstd;
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
  if (!args) return 0;
  const mma_residual_norm_backward_args r = in_use(*args);
  return check_join_backward(r, 0, nullptr, true, &d) == MMAEMU_OK ? join_plan(r).bytes : 0;
}

int mma_residual_norm_backward(const mma_residual_norm_backward_args* args, void* workspace,
                               int64_t workspace_bytes, void* hip_stream) {
  if (!args) return MMAEMU_ERR_NULL;
  const mma_residual_norm_backward_args r = in_use(*args);
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
  if (!plan.sums && !r.dX && !r.dbranch) return MMAEMU_OK;
  a.branch = r.branch;
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
  if (plan.sums) {
    a.partial = (float*)workspace;
    a.means = (float*)((char*)workspace + plan.means_at);
    a.spare = a.means;
  }
  err = MMAOPS_BY_TYPES(r.dtype, r.param_dtype, join_backward_launch, a, plan.groups, plan.shift,
                        s);
  if (err == hipSuccess && plan.sums) {
    const JoinSums j{a.partial, plan.groups, r.param_dtype, r.cols, r.gate, r.post_weight,
                     r.post_bias, r.post != kNormNone, r.dgate, r.dpost_weight, r.dpost_bias,
                     r.dpre_weight, r.dpre_bias};
    const int64_t blocks = (r.cols + 31) / 32;
    constexpr int64_t kMost = 1 << 20;
    const dim3 grid((uint32_t)(blocks < kMost ? blocks : kMost),
                    (uint32_t)((blocks + kMost - 1) / kMost));
    if (plan.shift)
      join_sums_kernel<true><<<grid, 1024, 0, s>>>(j);
    else
      join_sums_kernel<false><<<grid, 1024, 0, s>>>(j);
    err = hipGetLastError();
  }
  return err == hipSuccess ? MMAEMU_OK : hip_fail(err, "mma_residual_norm_backward launch");
}

int64_t mma_gated_linear_workspace(const mma_gated_linear_args* args) {
  if (!args || check_gated(*args, 0, nullptr, true) != MMAEMU_OK) return 0;
  return gated_need(*args);
}

int mma_gated_linear(const mma_gated_linear_args* args, void* workspace, int64_t workspace_bytes,
                     void* hip_stream) {
  if (!args) return MMAEMU_ERR_NULL;
  const mma_gated_linear_args& r = *args;
  const int rc = check_gated(r, workspace_bytes, workspace, false);
  if (rc || r.M == 0 || r.N == 0) return rc;
  const hipStream_t s = (hipStream_t)hip_stream;
  GateArgs g;
  memset(&g, 0, sizeof g);
  g.bias = r.bias_g;
  g.bias2 = r.bias_u;
  g.y = r.Y;
  g.ldy = r.ldy;
  g.z = r.G;
  g.ldz = r.ldg;
  g.z2 = r.U;
  g.ldz2 = r.ldu;
  g.codes = r.g_codes;
  g.scales = r.g_scales;
  g.codes2 = r.u_codes;
  g.scales2 = r.u_scales;
  g.bias_dt = r.bias_dtype;
  g.out_dt = r.out_dtype;
  g.act = r.activation;
  const Paired q = gated_product(r);
  const Plan plan = paired_plan(q, r.g_codes != nullptr);
  const void* a2;
  (void)hipGetLastError();
  hipError_t err = paired_fill(q, plan, g, a2, g.b2, workspace, s);
  if (err == hipSuccess) err = launches(r.dtype).gate(plan.tile, plan.direct, q.p.lb, g, s);
  return err == hipSuccess ? MMAEMU_OK : hip_fail(err, "mma_gated_linear launch");
}

int64_t mma_gated_linear_backward_workspace(const mma_gated_linear_backward_args* args) {
  if (!args || check_gated_backward(*args, 0, nullptr, true) != MMAEMU_OK) return 0;
  if (args->M == 0 || args->N == 0) return 0;
  return gated_backward(*args, nullptr).bytes;
}

int mma_gated_linear_backward(const mma_gated_linear_backward_args* args, void* workspace,
                              int64_t workspace_bytes, void* hip_stream) {
  if (!args) return MMAEMU_ERR_NULL;
  const int rc = check_gated_backward(*args, workspace_bytes, workspace, false);
  if (rc) return rc;
  const mma_gated_linear_backward_args& r = *args;
  if (!(r.dX && r.M && r.K) && !(r.dWg && r.K && r.N) && !((r.dbias_g || r.dbias_u) && r.N))
    return MMAEMU_OK;
  (void)hipGetLastError();
  const hipError_t err = gated_backward_run(r, workspace, (hipStream_t)hip_stream);
  return err == hipSuccess ? MMAEMU_OK : hip_fail(err, "mma_gated_linear_backward launch");
}

}  // extern "C"
