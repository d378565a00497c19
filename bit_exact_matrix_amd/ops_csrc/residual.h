// residual.h -- the sum of a block's output into the residual stream, with the
// norms after and before a block, forward and backward.
//
// Mathematics.  v = post(b), r = scale x + gate drop(v), h = pre(r).  A norm is
// a layer norm (norm.h), y = (x - mu) / sqrt(var + eps) w + bias, or an rms norm,
// the same with mu = 0.  Backward, with xh = (x - mu) rstd and q = dy w:
//   norm'(dy) = rstd (q - mean(q) - xh mean(q xh)), without mean(q) for rms
//   t = dr + pre'(dh);  dx = scale t;  db = post'(gate drop(t))
// and the vectors' gradients from four column sums over the rows,
//   p1 = sum dh rh, p0 = sum dh, s1 = sum drop(t) bh, s0 = sum drop(t):
//   dpre_w = p1, dpre_b = p0, dpost_w = gate s1, dpost_b = gate s0,
//   dgate = post_w s1 + post_b s0
// (bh = b where there is no post norm).  All in FP32; h is made from r as it
// is before r's rounding.
//
// One pass over the data: a row stays in its lanes' registers from the loads to
// the stores, and the next row's loads are under way meanwhile.  Bound by memory
// (one MI355X, 8192 x 4096 bf16, both rms norms, gate, dropout): forward 53 us for
// 268 MB, 5.0 TB/s (197 where a row is read for each of its sums), backward 81 for
// 403 MB, 5.0 TB/s, and 6.4 for the sums of the workgroups' partial rows (239 and 71).
// Layer norms: 57, and 87 and 9.  FP32 (537 and 805 MB): forward 105, backward 148 and 5.
//
// What does not fit the registers.  A CU's 16 waves have 128 a lane each.  FP32
// vectors beside 16-bit matrices, in rows of two vectors a lane forward, take 80 for the
// vectors alone (2048 x 16384 177 us; vectors in 16 bits 62; one vector a lane, 4096 x
// 8192, 69 and 62), and backward rows of 9 to 16 waves with biases hold four sums beside
// their four matrices (4096 x 8192 bf16 169 us, without biases 82; 3276 x 5120 FP32, 8
// elements a lane, 180 and 122).  There the compiler spills up to 101 registers, whose
// loads the waits for a row's loads then count too.
#ifndef MMAOPS_RESIDUAL_H
#define MMAOPS_RESIDUAL_H

#include "random.h"

namespace mmaops {

enum { kNormNone = 0, kNormLayer = 1, kNormRms = 2 };

struct JoinArgs {
  const void* x;
  const void* branch;
  int64_t ldx, ldb;
  const void *gate, *post_w, *post_b, *pre_w, *pre_b;  // or NULL each
  void* r;  // backward: the forward pass's, read
  void* h;
  int64_t ldr, ldh;
  float *post_mean, *post_rstd, *mean, *rstd;
  int64_t rows;
  int cols, post, pre;
  float scale, eps;
  DropArgs drop;
  // backward
  const void *dr, *dh;
  void *dx, *db;
  int64_t lddr, lddh, lddx, lddb;
  float* partial;  // [groups][4][cols]: p1, p0, s1, s0
  float* means;    // long rows: [rows][2], the means of pre'
  void* spare;     // where neither dx nor db is wanted: a row for each at work
};

// V elements of a parameter at column c, `fill` where there is none
template <int PDT, int V>
__device__ __forceinline__ void param(const void* p, int c, int n, float fill, float (&v)[V]) {
  if (p && n > 0) {
    unpack(load_pack<PDT, V>((const elem_t<PDT>*)p + c, n), v);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = fill;
  }
}

// --------------------------------------------------- rows of any length
// One workgroup a row, the row read again for each of its sums.  2048 x 16384, what
// has to be read and written once: backward bf16 161 us for both inputs' gradients and
// 66 for the vectors', 1.8 TB/s, FP32 271 and 126; forward FP32 213, 2.5 TB/s (1024 x
// 32768 bf16 120).

// Mean and rstd of a row whose elements fn(c, n, v) gives, 0 past its end.
template <int GT, int V, typename FN>
__device__ __forceinline__ void row_stats(FN fn, int cols, bool layer, float eps, float* lds,
                                          int& turn, float& mean, float& rstd) {
  const float n_f = (float)cols;
  float s[1], mu = 0.0f;
  if (layer) {
    s[0] = 0.0f;
    for (int c = threadIdx.x * V; c < cols; c += GT * V) {
      float v[V];
      fn(c, cols - c, v);
      s[0] += pair_sum(v);
    }
    row_sum<GT, 1>(s, lds, turn);
    mu = s[0] / n_f;
  }
  auto centred = [&](bool square) {
    s[0] = 0.0f;
    for (int c = threadIdx.x * V; c < cols; c += GT * V) {
      float v[V];
      fn(c, cols - c, v);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[i] = c + i < cols ? v[i] - mu : 0.0f;
        if (square) v[i] *= v[i];
      }
      s[0] += pair_sum(v);
    }
    row_sum<GT, 1>(s, lds, turn);
    return s[0] / n_f;
  };
  float var = centred(true);
  mean = mu;
  if (layer && row_far(mu, var, eps)) row_correct(centred(false), mean, var);
  rstd = 1.0f / sqrtf(var + eps);
}

template <int DT, int PDT>
__global__ __launch_bounds__(1024) void join_long_kernel(JoinArgs a) {
  constexpr int V = kVec<DT>, GT = 1024;
  using E = elem_t<DT>;
  __shared__ float lds[2 * 16];
  int turn = 0;
  const Drop drop(a.drop);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const E* const x = (const E*)a.x + row * a.ldx;
    const E* const b = (const E*)a.branch + row * a.ldb;
    float pm = 0.0f, pr = 1.0f, m = 0.0f, q = 1.0f;
    if (a.post != kNormNone)
      row_stats<GT, V>([&](int c, int n, float (&v)[V]) { unpack(load_pack<DT, V>(b + c, n), v); },
                       a.cols, a.post == kNormLayer, a.eps, lds, turn, pm, pr);
    auto sum = [&](int c, int n, float (&v)[V]) {
      float t[V], u[V];
      unpack(load_pack<DT, V>(b + c, n), v);
      if (a.post != kNormNone) {
        param<PDT, V>(a.post_w, c, n, 1.0f, t);
        param<PDT, V>(a.post_b, c, n, 0.0f, u);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = (v[i] - pm) * pr * t[i] + u[i];
      }
      if (drop.threshold) {
        uint32_t w[V / 2];
        drop.halves<V>(row, c, w);
        drop.apply<V>(w, v);
      }
      param<PDT, V>(a.gate, c, n, 1.0f, t);
      unpack(load_pack<DT, V>(x + c, n), u);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = i < n ? u[i] * a.scale + t[i] * v[i] : 0.0f;
    };
    if (a.pre != kNormNone)
      row_stats<GT, V>(sum, a.cols, a.pre == kNormLayer, a.eps, lds, turn, m, q);
    for (int c = threadIdx.x * V; c < a.cols; c += GT * V) {
      const int n = a.cols - c;
      float v[V], w[V], u[V];
      sum(c, n, v);
      store_pack<DT, V>((E*)a.r + row * a.ldr + c, pack<DT, V>(v), n);
      if (a.pre == kNormNone) continue;
      param<PDT, V>(a.pre_w, c, n, 1.0f, w);
      param<PDT, V>(a.pre_b, c, n, 0.0f, u);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = (v[i] - m) * q * w[i] + u[i];
      store_pack<DT, V>((E*)a.h + row * a.ldh + c, pack<DT, V>(v), n);
    }
    if (threadIdx.x == 0) {
      if (a.post_mean) a.post_mean[row] = pm;
      if (a.post_rstd) a.post_rstd[row] = pr;
      if (a.mean) a.mean[row] = m;
      if (a.rstd) a.rstd[row] = q;
    }
  }
}

// What the backward pass knows of a row before its sums.
struct JoinRow {
  float pm, pr, m, q;  // statistics
  __device__ __forceinline__ JoinRow(const JoinArgs& a, int64_t row) {
    pm = a.post == kNormLayer ? a.post_mean[row] : 0.0f;
    pr = a.post != kNormNone ? a.post_rstd[row] : 1.0f;
    m = a.pre == kNormLayer ? a.mean[row] : 0.0f;
    q = a.pre != kNormNone ? a.rstd[row] : 1.0f;
  }
};

// dh, rh = (r - m) q and t = dr + pre'(dh) of V columns, 0 past the row's
// end; m0 and m1 are the means of dh w and of dh w rh.
template <int DT, int PDT, int V>
__device__ __forceinline__ void join_t(const JoinArgs& a, const JoinRow& s, int64_t row, int c,
                                       int n, float m0, float m1, float (&dh)[V], float (&rh)[V],
                                       float (&t)[V]) {
  using E = elem_t<DT>;
  if (a.dr) {
    unpack(load_pack<DT, V>((const E*)a.dr + row * a.lddr + c, n), t);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) t[i] = 0.0f;
  }
  if (a.pre == kNormNone) return;
  float w[V];
  unpack(load_pack<DT, V>((const E*)a.dh + row * a.lddh + c, n), dh);
  unpack(load_pack<DT, V>((const E*)a.r + row * a.ldr + c, n), rh);
  param<PDT, V>(a.pre_w, c, n, 1.0f, w);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    rh[i] = i < n ? (rh[i] - s.m) * s.q : 0.0f;
    if (i < n) t[i] += s.q * (dh[i] * w[i] - m0 - rh[i] * m1);
  }
}

// drop(t), and bh = (b - pm) pr where the branch is read.  For the column sums
// bh is 0 where it was dropped, whatever it was: without a post norm an
// infinity there has no part in the gate's gradient.
template <int DT, int V, bool SUMS>
__device__ __forceinline__ void join_branch(const JoinArgs& a, const JoinRow& s, const Drop& drop,
                                            int64_t row, int c, int n, float (&t)[V],
                                            float (&bh)[V]) {
  if (a.branch) {
    unpack(load_pack<DT, V>((const elem_t<DT>*)a.branch + row * a.ldb + c, n), bh);
#pragma unroll
    for (int i = 0; i < V; ++i) bh[i] = i < n ? (bh[i] - s.pm) * s.pr : 0.0f;
  }
  if (drop.threshold) {
    uint32_t w[V / 2];
    drop.halves<V>(row, c, w);
    drop.apply<V>(w, t);
    if (SUMS) drop.clear<V>(w, bh);
  }
}

template <int DT, int PDT>
__global__ __launch_bounds__(1024) void join_long_dx_kernel(JoinArgs a) {
  constexpr int V = kVec<DT>, GT = 1024;
  using E = elem_t<DT>;
  __shared__ float lds[2 * 16 * 2];
  int turn = 0;
  const Drop drop(a.drop);
  const float n_f = (float)a.cols;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const JoinRow st(a, row);
    float s[2] = {0.0f, 0.0f}, m0 = 0.0f, m1 = 0.0f, k0 = 0.0f, k1 = 0.0f;
    if (a.pre != kNormNone) {
      for (int c = threadIdx.x * V; c < a.cols; c += GT * V) {
        const int n = a.cols - c;
        float dh[V], rh[V], w[V];
        unpack(load_pack<DT, V>((const E*)a.dh + row * a.lddh + c, n), dh);
        unpack(load_pack<DT, V>((const E*)a.r + row * a.ldr + c, n), rh);
        param<PDT, V>(a.pre_w, c, n, 1.0f, w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          rh[i] = i < n ? (rh[i] - st.m) * st.q : 0.0f;
          dh[i] *= w[i];
          rh[i] *= dh[i];
        }
        s[0] += pair_sum(dh);
        s[1] += pair_sum(rh);
      }
      row_sum<GT, 2>(s, lds, turn);
      m0 = a.pre == kNormLayer ? s[0] / n_f : 0.0f;
      m1 = s[1] / n_f;
    }
    if (a.means && threadIdx.x == 0) {
      a.means[row * 2] = m0;
      a.means[row * 2 + 1] = m1;
    }
    // q = drop(t) gate w and bh of a vector
    auto inner = [&](int c, int n, float (&t)[V], float (&q)[V], float (&bh)[V]) {
      float dh[V], rh[V], g[V], w[V];
      join_t<DT, PDT, V>(a, st, row, c, n, m0, m1, dh, rh, t);
#pragma unroll
      for (int i = 0; i < V; ++i) q[i] = t[i];
      join_branch<DT, V, false>(a, st, drop, row, c, n, q, bh);
      param<PDT, V>(a.gate, c, n, 1.0f, g);
      param<PDT, V>(a.post_w, c, n, 1.0f, w);
#pragma unroll
      for (int i = 0; i < V; ++i) q[i] = i < n ? q[i] * g[i] * w[i] : 0.0f;
    };
    if (a.post != kNormNone && a.db) {
      s[0] = s[1] = 0.0f;
      for (int c = threadIdx.x * V; c < a.cols; c += GT * V) {
        float t[V], q[V], bh[V];
        inner(c, a.cols - c, t, q, bh);
#pragma unroll
        for (int i = 0; i < V; ++i) bh[i] *= q[i];
        s[0] += pair_sum(q);
        s[1] += pair_sum(bh);
      }
      row_sum<GT, 2>(s, lds, turn);
      k0 = a.post == kNormLayer ? s[0] / n_f : 0.0f;
      k1 = s[1] / n_f;
    }
    if (!a.dx && !a.db) continue;
    for (int c = threadIdx.x * V; c < a.cols; c += GT * V) {
      const int n = a.cols - c;
      float t[V], q[V], bh[V];
      inner(c, n, t, q, bh);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (a.post != kNormNone) q[i] = st.pr * (q[i] - k0 - bh[i] * k1);
        t[i] *= a.scale;
      }
      if (a.dx) store_pack<DT, V>((E*)a.dx + row * a.lddx + c, pack<DT, V>(t), n);
      if (a.db) store_pack<DT, V>((E*)a.db + row * a.lddb + c, pack<DT, V>(q), n);
    }
  }
}

// Partial column sums over a run of rows, for the columns of one workgroup
// (64 lanes of V columns each, four waves over the rows).
template <int DT, int PDT>
__global__ __launch_bounds__(256) void join_long_sums_kernel(JoinArgs a, int64_t run) {
  constexpr int V = kVec<DT>;
  __shared__ float meet[4][4][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = (blockIdx.x * 64 + lane) * V, n = a.cols - c;
  const int64_t r0 = blockIdx.y * run, r1 = r0 + run < a.rows ? r0 + run : a.rows;
  const Drop drop(a.drop);
  float sum[4][V];
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) sum[k][i] = 0.0f;
  if (n > 0)
    for (int64_t row = r0 + wave; row < r1; row += 4) {
      const JoinRow st(a, row);
      float dh[V], rh[V], t[V], bh[V];
#pragma unroll
      for (int i = 0; i < V; ++i) dh[i] = rh[i] = bh[i] = 0.0f;
      join_t<DT, PDT, V>(a, st, row, c, n, a.means[row * 2], a.means[row * 2 + 1], dh, rh, t);
      join_branch<DT, V, true>(a, st, drop, row, c, n, t, bh);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        sum[0][i] += dh[i] * rh[i];
        sum[1][i] += dh[i];
        sum[2][i] += t[i] * bh[i];
        sum[3][i] += t[i];
      }
    }
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) meet[k][wave][i * 64 + lane] = sum[k][i];
  __syncthreads();
  float* const out = a.partial + ((int64_t)blockIdx.y * 4 + wave) * a.cols;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float s = 0.0f;
    for (int q = 0; q < 4; ++q) s += meet[wave][q][i * 64 + lane];
    if (i < n) out[c + i] = s;
  }
}

// ------------------------------------------------------ rows in registers
// A row is held by whole waves, no more than it needs: W of them where a
// workgroup has G > 1 rows (or W = 1), up to W where it has one, as many as the
// workgroup has.  (Powers of two of waves left lanes idle, and bytes in flight with
// them: 13107 x 2560 bf16 forward 78 us, this way 58; 6553 x 5120 backward 136 and 91.)
template <int W, int G>
__device__ __forceinline__ int row_lanes() {
  return G > 1 || W == 1 ? W * 64 : (int)blockDim.x;
}

// Sums of N values over a row's waves, the same in each of its lanes, as row_sum
// has them.  `lds` has 2 * 16 * N floats, zeros at first: those of waves that
// are not there stay zero.
template <int N>
__device__ __forceinline__ void join_sum_start(float* lds) {
  if (threadIdx.x < 2 * 16 * N) lds[threadIdx.x] = 0.0f;
  __syncthreads();
}
template <int W, int G, int N>
__device__ __forceinline__ void join_sum(float (&v)[N], float* lds, int& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (W > 1) {
    float* const buf = lds + turn * 16 * N;
    turn ^= 1;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) buf[wave * N + i] = v[i];
    }
    __syncthreads();
    const int first = G > 1 ? wave / W * W : 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += buf[(first + w) * N + i];
      v[i] = s;
    }
  }
}

// A parameter's vectors as they are in memory, for all of a lane's columns.
template <int PDT, int V, int NV>
struct Vectors {
  Pack<PDT, V> q[NV];
  __device__ __forceinline__ void load(const void* p, int lane, int lanes, int cols, float fill) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * lanes + lane) * V;
      float v[V];
      param<PDT, V>(p, c, cols - c, fill, v);
      q[j] = pack<PDT, V>(v);
    }
  }
  // Two vectors a lane: unpacked where they are used, in every row; taken out of
  // the loop they would hold twice the registers.  One: unpacked once (the forward
  // pass of 8192 x 4096 bf16 54 us, in every row 59).
  __device__ __forceinline__ void values(int j, float (&v)[V]) {
    if constexpr (NV > 1) hide(q[j]);
    unpack(q[j], v);
  }
};

// Mean and rstd of a row held by its lanes, NV vectors each, which are centred
// on the way (0 past the row's end).  As in norm_kernel.
template <int W, int G, int NV, int V>
__device__ __forceinline__ void held_stats(float (&v)[NV][V], int lane, int lanes, int cols,
                                           bool layer, float eps, float* lds, int& turn, float& mean,
                                           float& rstd) {
  const float n_f = (float)cols;
  float s[1], mu = 0.0f;
  if (layer) {
    s[0] = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) s[0] += pair_sum(v[j]);
    join_sum<W, G, 1>(s, lds, turn);
    mu = s[0] / n_f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int n = cols - (j * lanes + lane) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) v[j][i] = i < n ? v[j][i] - mu : 0.0f;
    }
  }
  s[0] = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float t[V];
#pragma unroll
    for (int i = 0; i < V; ++i) t[i] = v[j][i] * v[j][i];
    s[0] += pair_sum(t);
  }
  join_sum<W, G, 1>(s, lds, turn);
  float var = s[0] / n_f;
  mean = mu;
  // the same in all lanes that meet at its barriers
  if (layer && row_far(mu, var, eps)) {
    s[0] = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) s[0] += pair_sum(v[j]);
    join_sum<W, G, 1>(s, lds, turn);
    const float d = s[0] / n_f;
    row_correct(d, mean, var);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) v[j][i] -= d;
  }
  rstd = 1.0f / sqrtf(var + eps);
}

// A lane has NV vectors of 16 bytes of each matrix's row; a workgroup works on
// G rows at a time (several only where a row is a wave) and walks the matrices,
// the next rows' loads under way.  (FP32 vectors beside 16-bit matrices: see above
// for what they take.)
template <int DT, int PDT, int W, int NV, int G>
__global__ __launch_bounds__(W * 64 * G, NV == 1 ? 5 : 4) void join_kernel(JoinArgs a) {
  constexpr int V = kVec<DT>;
  using E = elem_t<DT>;
  static_assert(G == 1 || W == 1, "");
  __shared__ float lds[2 * 16];
  const int lanes = row_lanes<W, G>();
  const int lane = G > 1 ? threadIdx.x % (W * 64) : threadIdx.x;
  const int g = G > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / (W * 64)) : 0;
  join_sum_start<1>(lds);
  int turn = 0;
  const Drop drop(a.drop);
  Vectors<PDT, V, NV> gate, post_w, post_b, pre_w, pre_b;
  gate.load(a.gate, lane, lanes, a.cols, 1.0f);
  post_w.load(a.post_w, lane, lanes, a.cols, 1.0f);
  post_b.load(a.post_b, lane, lanes, a.cols, 0.0f);
  pre_w.load(a.pre_w, lane, lanes, a.cols, 1.0f);
  pre_b.load(a.pre_b, lane, lanes, a.cols, 0.0f);
  const int64_t step = (int64_t)gridDim.x * G;
  Pack<DT, V> xr[NV], br[NV];
  auto fetch = [&](int64_t row) {
    const bool live = row < a.rows;
    const E* const x = (const E*)a.x + (live ? row : 0) * a.ldx;
    const E* const b = (const E*)a.branch + (live ? row : 0) * a.ldb;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * lanes + lane) * V;
      br[j] = load_pack<DT, V>(b + c, live ? a.cols - c : 0);
      xr[j] = load_pack<DT, V>(x + c, live ? a.cols - c : 0);
    }
  };
  int64_t r0 = (int64_t)blockIdx.x * G;
  fetch(r0 + g);
  for (; r0 < a.rows; r0 += step) {
    const int64_t row = r0 + g;
    const bool live = row < a.rows;
    float v[NV][V];
    Pack<DT, V> x[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      unpack(br[j], v[j]);
      x[j] = xr[j];
    }
    if (r0 + step < a.rows) fetch(row + step);
    float pm = 0.0f, pr = 1.0f, m = 0.0f, q = 1.0f;
    if (a.post != kNormNone) {
      held_stats<W, G, NV, V>(v, lane, lanes, a.cols, a.post == kNormLayer, a.eps, lds, turn, pm, pr);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float w[V], b[V];
        post_w.values(j, w);
        post_b.values(j, b);
#pragma unroll
        for (int i = 0; i < V; ++i) v[j][i] = v[j][i] * pr * w[i] + b[i];
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * lanes + lane) * V;
      if (drop.threshold) {
        uint32_t w[V / 2];
        drop.halves<V>(row, c, w);
        drop.apply<V>(w, v[j]);
      }
      float k[V], t[V];
      gate.values(j, k);
      unpack(x[j], t);
#pragma unroll
      for (int i = 0; i < V; ++i) v[j][i] = t[i] * a.scale + k[i] * v[j][i];
      if (live) store_pack<DT, V>((E*)a.r + row * a.ldr + c, pack<DT, V>(v[j]), a.cols - c);
    }
    if (a.pre != kNormNone) {
      // past the row's end there may be a bias by now
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int n = a.cols - (j * lanes + lane) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) v[j][i] = i < n ? v[j][i] : 0.0f;
      }
      held_stats<W, G, NV, V>(v, lane, lanes, a.cols, a.pre == kNormLayer, a.eps, lds, turn, m, q);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * lanes + lane) * V;
        float w[V], b[V];
        pre_w.values(j, w);
        pre_b.values(j, b);
#pragma unroll
        for (int i = 0; i < V; ++i) v[j][i] = v[j][i] * q * w[i] + b[i];
        if (live) store_pack<DT, V>((E*)a.h + row * a.ldh + c, pack<DT, V>(v[j]), a.cols - c);
      }
    }
    if (live && lane == 0) {
      if (a.post_mean) a.post_mean[row] = pm;
      if (a.post_rstd) a.post_rstd[row] = pr;
      if (a.mean) a.mean[row] = m;
      if (a.rstd) a.rstd[row] = q;
    }
  }
}

// The gradients of x and of the branch, and the workgroup's part of the
// column sums (SHIFT: p0 and s0 too, which only biases need): V elements a lane,
// G rows at a time (WHOLE: all of a row's lanes have them).  What a row's sums need is made again from the
// loaded elements after they have met.  Each matrix's next row is loaded as soon as
// this one's has been used, with no registers of its own.  An element past a
// row's end adds 0 to the row's sums: its dh and rh are 0 in the first ones, its
// gate post_w t and b in the second.
template <int DT, int PDT, int V, int W, int G, bool SHIFT, bool WHOLE>
__global__ __launch_bounds__(W * 64 * G, 4) void join_backward_kernel(JoinArgs a) {
  using E = elem_t<DT>;
  __shared__ float lds[2 * 16 * 2];
  const int lane = G > 1 ? threadIdx.x % (W * 64) : threadIdx.x;
  const int g = G > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / (W * 64)) : 0;
  join_sum_start<2>(lds);
  const int c = lane * V, n = WHOLE ? V : a.cols - c;
  int turn = 0;
  const Drop drop(a.drop);
  float pre_w[V], inner_w[V];  // inner_w: gate post_w, 0 past the row's end
  param<PDT, V>(a.pre_w, c, n, 1.0f, pre_w);
  {
    float k[V];
    param<PDT, V>(a.post != kNormNone ? a.post_w : nullptr, c, n, 1.0f, inner_w);
    param<PDT, V>(a.gate, c, n, 1.0f, k);
#pragma unroll
    for (int i = 0; i < V; ++i) inner_w[i] = i < n ? inner_w[i] * k[i] : 0.0f;
  }
  float p1[V], p0[V], s1[V], s0[V];
#pragma unroll
  for (int i = 0; i < V; ++i) p1[i] = p0[i] = s1[i] = s0[i] = 0.0f;
  const float n_f = (float)a.cols;
  const int64_t step = (int64_t)gridDim.x * G;

  // A row's loads, and the store of dx, are there whatever is asked for: a matrix
  // that is not has another in its place, whose row is in the cache, and dx, if it
  // is not wanted, goes where the branch's gradient will be written over it, or to
  // spare rows.  Behind a branch they could not be counted, and the wait for a
  // row's loads would be one for the stores behind them (8192 x 4096 bf16, both rms
  // norms, gate, dropout: that way 95 us, this way 81).
  const void* const dr_p = a.dr ? a.dr : a.dh;
  const int64_t dr_ld = a.dr ? a.lddr : a.lddh;
  const void* const dh_p = a.pre != kNormNone ? a.dh : dr_p;
  const int64_t dh_ld = a.pre != kNormNone ? a.lddh : dr_ld;
  const void* const r_p = a.pre != kNormNone ? a.r : dr_p;
  const int64_t r_ld = a.pre != kNormNone ? a.ldr : dr_ld;
  const void* const b_p = a.branch ? a.branch : dr_p;
  const int64_t b_ld = a.branch ? a.ldb : dr_ld;
  E* const dx_p = a.dx   ? (E*)a.dx
                  : a.db ? (E*)a.db
                         : (E*)a.spare + ((int64_t)blockIdx.x * G + g) * a.cols;
  const int64_t dx_ld = a.dx ? a.lddx : a.db ? a.lddb : 0;
  Pack<DT, V> dh, rr, dr, br;
  float pm, pr, m, rs;
  auto load = [&](const void* p, int64_t ld, int64_t row, int k) {
    const E* const at = (const E*)p + row * ld;
    if constexpr (WHOLE) return load_pack<DT, V>(at + c);
    return load_pack<DT, V>(at + c, k);
  };
  auto fetch = [&](int64_t row) {
    const bool live = row < a.rows;
    const int64_t at = live ? row : a.rows - 1;
    const int k = live ? n : 0;
    br = load(b_p, b_ld, at, k);
    dr = load(dr_p, dr_ld, at, k);
    dh = load(dh_p, dh_ld, at, k);
    rr = load(r_p, r_ld, at, k);
    m = a.pre == kNormLayer ? a.mean[at] : 0.0f;
    rs = a.pre != kNormNone ? a.rstd[at] : 1.0f;
    pm = a.post == kNormLayer ? a.post_mean[at] : 0.0f;
    pr = a.post != kNormNone ? a.post_rstd[at] : 1.0f;
  };
  // A row past the end has another's elements and statistics, which may be no
  // numbers, and an element past a row's end is the row's mean below 0, in t that of
  // dh w, which its rstd may take past a float: they are cleared, and not multiplied
  // with 0.  t is cleared where it enters a sum: before, rows of 5000 elements with
  // biases took 190 us for 173 in FP32 and 196 for 225 in bf16, by the registers that
  // the compiler then spills (without the 0 of inner_w 188 and 227).
  auto none = [](float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.0f;
  };
  auto only = [&](float (&v)[V], bool live) {
    if (G > 1 && !live) none(v);
    if (WHOLE) return;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = i < n ? v[i] : 0.0f;
  };
  int64_t row = (int64_t)blockIdx.x * G + g;
  fetch(row);
  // every group of the workgroup takes as many turns (rows past the end
  // are empty), for the barriers
  for (int64_t r0 = (int64_t)blockIdx.x * G; r0 < a.rows; r0 += step, row += step) {
    const bool live = G == 1 || row < a.rows;
    float s[2], t[V], b[V];
    if (a.pre != kNormNone) {
      float rh[V], h[V], d[V];
      unpack(rr, rh);
      unpack(dh, d);
#pragma unroll
      for (int i = 0; i < V; ++i) rh[i] = (rh[i] - m) * rs;
      if (G > 1 && !live) none(d);
      only(rh, live);
      s[0] = s[1] = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        h[i] = d[i] * pre_w[i];
        s[0] += h[i];
        s[1] += h[i] * rh[i];
        p1[i] += d[i] * rh[i];
        if (SHIFT) p0[i] += d[i];
      }
      join_sum<W, G, 2>(s, lds, turn);
      const float m0 = a.pre == kNormLayer ? s[0] / n_f : 0.0f, m1 = s[1] / n_f;
      unpack(dr, t);
#pragma unroll
      for (int i = 0; i < V; ++i) t[i] = (a.dr ? t[i] : 0.0f) + rs * (h[i] - m0 - rh[i] * m1);
    } else {
      unpack(dr, t);
    }
    unpack(br, b);
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = (b[i] - pm) * pr;
    if (G > 1 && !live) none(t);
    only(b, live);
    const float pr_now = pr;
    if (r0 + step < a.rows) fetch(row + step);
    if (live) {
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = t[i] * a.scale;
      store_pack<DT, V>(dx_p + row * dx_ld + c, pack<DT, V>(o), n);
    }
    if (drop.threshold) {
      uint32_t w[V / 2];
      drop.halves<V>(row, c, w);
      drop.apply<V>(w, t);
      float k[V];
#pragma unroll
      for (int i = 0; i < V; ++i) k[i] = b[i];
      drop.clear<V>(w, k);  // what was dropped has no part, whatever it was
#pragma unroll
      for (int i = 0; i < V; ++i) s1[i] += t[i] * k[i];
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) s1[i] += t[i] * b[i];
    }
    if (SHIFT) {
#pragma unroll
      for (int i = 0; i < V; ++i) s0[i] += t[i];
    }
    if (!a.db) continue;
#pragma unroll
    for (int i = 0; i < V; ++i) t[i] = WHOLE || i < n ? t[i] * inner_w[i] : 0.0f;
    if (a.post != kNormNone) {
      s[0] = s[1] = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[0] += t[i];
        s[1] += t[i] * b[i];
      }
      join_sum<W, G, 2>(s, lds, turn);
      const float k0 = a.post == kNormLayer ? s[0] / n_f : 0.0f, k1 = s[1] / n_f;
#pragma unroll
      for (int i = 0; i < V; ++i) t[i] = pr_now * (t[i] - k0 - b[i] * k1);
    }
    if (live) store_pack<DT, V>((E*)a.db + row * a.lddb + c, pack<DT, V>(t), n);
  }
  if (!a.partial) return;
  float* const out = a.partial + (int64_t)blockIdx.x * 4 * a.cols;
  float(*const sums[4])[V] = {&p1, &p0, &s1, &s0};
  if constexpr (G == 1) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (SHIFT || k % 2 == 0)
        store_pack<kFP32, V>(out + k * a.cols + c, pack<kFP32, V>(*sums[k]), n);
  } else {  // the G rows' sums meet in LDS, in group order
    constexpr int GT = W * 64;
    __shared__ float meet[G][GT * V];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (!SHIFT && k % 2) continue;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < V; ++i) meet[g][i * GT + lane] = (*sums[k])[i];
      __syncthreads();
      for (int t = threadIdx.x; t < GT * V; t += GT * G) {
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < G; ++q) s += meet[q][(t % V) * GT + t / V];
        if (t < a.cols) out[(int64_t)k * a.cols + t] = s;
      }
    }
  }
}

// -------------------------------------------------- the vectors' gradients
struct JoinSums {
  const float* partial;  // [count][4][cols]
  int count, dt;
  int64_t cols;
  const void *gate, *post_w, *post_b;
  bool post;
  void *dgate, *dpost_w, *dpost_b, *dpre_w, *dpre_b;
};

// The groups' sums in group order within each of 32 runs and then in run
// order: 32 columns a workgroup.  SHIFT: p0 and s0 are there.
template <bool SHIFT>
__global__ __launch_bounds__(1024) void join_sums_kernel(JoinSums a) {
  __shared__ float meet[4][32][32], total[4][32];
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  // a grid has fewer than 2^32 lanes in x: the longest rows take several of it
  const int64_t c = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 32 + lane;
  const int run = (a.count + 31) / 32;
  const int p0 = part * run, p1 = p0 + run < a.count ? p0 + run : a.count;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < a.cols) {
    const float* const p = a.partial + c;
#pragma unroll 8
    for (int q = p0; q < p1; ++q)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (SHIFT || k % 2 == 0) s[k] += p[((int64_t)q * 4 + k) * a.cols];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) meet[k][part][lane] = s[k];
  __syncthreads();
  if (part < 4) {
    float t = meet[part][0][lane];
#pragma unroll
    for (int w = 1; w < 32; ++w) t += meet[part][w][lane];
    total[part][lane] = t;
  }
  __syncthreads();
  if (part || c >= a.cols) return;
#pragma unroll
  for (int k = 0; k < 4; ++k) s[k] = total[k][lane];
  const float g = a.gate ? load_any(a.gate, c, a.dt) : 1.0f;
  if (a.dpre_w) store_any(a.dpre_w, c, s[0], a.dt);
  if (a.dpre_b) store_any(a.dpre_b, c, s[1], a.dt);
  if (a.dpost_w) store_any(a.dpost_w, c, g * s[2], a.dt);
  if (a.dpost_b) store_any(a.dpost_b, c, g * s[3], a.dt);
  if (a.dgate) {
    const float w = a.post && a.post_w ? load_any(a.post_w, c, a.dt) : 1.0f;
    const float b = a.post && a.post_b ? load_any(a.post_b, c, a.dt) : 0.0f;
    store_any(a.dgate, c, w * s[2] + b * s[3], a.dt);
  }
}

}  // namespace mmaops
#endif
