// norm.h -- layer norm of the rows of a matrix, forward and backward, and
// the reduction of the weight's and the bias's gradient.
//
// Mathematics.  mu = sum x / n, r = 1 / sqrt(sum (x - mu)^2 / n + eps), the
// second sum over the centred values (a difference of two large sums would
// lose what the row's offset holds).  mu is off by a few roundings of itself,
// which r makes large where the offset is large beside the spread (of a row
// of equal values it leaves a spread where there is none): there a third sum
// corrects it.  Backward, with xh = (x - mu) r and
// h = dy w: dx = r (h - sum h / n - xh sum(h xh) / n), dw = sum over rows of
// dy xh, db = sum over rows of dy.  All in FP32.
//
// What bounds both is memory: each element is read once and written once,
// and a row stays in registers between its sums and its output.  A row is
// held by GT lanes, NV vectors of 16 bytes each (one, as long as 1024 lanes
// are enough: two cost the backward pass its registers, 134 us against 55
// at 8192 x 4096 bf16); a workgroup of GT * G lanes works on G rows at a
// time and walks the matrix, so weight and bias are loaded once and the
// weight gradient's sums stay in registers until the workgroup's last row.
// Each workgroup then writes one row of partial sums, and a second kernel
// adds those in workgroup order: the result does not depend on which
// workgroup ran first.
//
// Measured, 8192 x 4096 bf16 (medians): forward 26 us (134 MB, 5.2 TB/s), with
// the checkpoint 32 us (169 MB, 5.3 TB/s); backward 42 us (201 MB, 4.8 TB/s) and
// 4.8 us for the partial sums.  A copy of 256 MiB reaches 5.4 TB/s.
#ifndef MMAOPS_NORM_H
#define MMAOPS_NORM_H

#include "ops_common.h"

namespace mmaops {

template <int DT>
constexpr int kVec = 16 / (DT == kFP32 ? 4 : 2);  // elements of a 16-byte vector

// Sums of N values over the GT lanes of a row, the same in each of them.
// `lds` has 2 * 16 * N floats: two buffers that calls use in turn, so that
// one barrier a call is enough (a lane can write a buffer again only after
// the barrier of the call between, which every reader of it has reached).
template <int GT, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* lds, int& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (GT > 64) {
    constexpr int W = GT / 64;
    float* const buf = lds + turn * 16 * N;
    turn ^= 1;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) buf[wave * N + i] = v[i];
    }
    __syncthreads();
    const int first = wave / W * W;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += buf[(first + w) * N + i];
      v[i] = s;
    }
  }
}

// A row whose mean is more than four times its spread, var + eps: its mean is
// corrected by d = mean (x - mu), and the variance by d^2.  Below, mu's error
// moves y by a few times 4 * 2^-24.  (For every row: the forward pass of 8192
// x 4096 bf16 with checkpoint took 36 us, so 32.)
__device__ __forceinline__ bool row_far(float mu, float var, float eps) {
  return mu * mu > 16.0f * (var + eps);
}
__device__ __forceinline__ void row_correct(float d, float& mu, float& var) {
  mu += d;
  var = __builtin_fmaf(-d, d, var);
  var = var < 0.0f ? 0.0f : var;  // keeps NaN
}

struct NormArgs {
  const void* x;
  int64_t ldx;
  const uint8_t* codes;  // backward: the checkpoint in x's place
  const uint8_t* scales;
  const void* weight;
  const void* bias;
  void* y;
  int64_t ldy;
  float* mean;
  float* rstd;
  uint8_t* codes_out;
  uint8_t* scales_out;
  int64_t rows;
  int cols;
  float eps;
  // backward
  const void* dy;
  int64_t lddy;
  float* partial;  // [gridDim.x][2][cols]
};

// weight or bias of a lane's vectors, `fill` where there is none
template <int PDT, int V, int NV, int GT>
__device__ __forceinline__ void load_param(const void* p, int lane, int cols, float fill,
                                           float (&v)[NV][V]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * GT + lane) * V;
    const int n = cols - c;
    if (p && n > 0) {
      unpack(load_pack<PDT, V>((const elem_t<PDT>*)p + c, n), v[j]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[j][i] = fill;
    }
  }
}

template <int DT, int PDT, int GT, int NV, int G, bool SAVE>
__global__ __launch_bounds__(GT* G) void norm_kernel(NormArgs a) {
  constexpr int V = kVec<DT>;
  using E = elem_t<DT>;
  __shared__ float lds[2 * 16];
  const int lane = threadIdx.x % GT, g = threadIdx.x / GT;
  int turn = 0;
  float w[NV][V], b[NV][V];
  load_param<PDT, V, NV, GT>(a.weight, lane, a.cols, 1.0f, w);
  load_param<PDT, V, NV, GT>(a.bias, lane, a.cols, 0.0f, b);
  const float n_f = (float)a.cols;
  const int64_t step = (int64_t)gridDim.x * G;
  // the next rows' loads are in flight while this row's sums meet
  Pack<DT, V> raw[NV];
  auto fetch = [&](int64_t row) {
    const E* const x = (const E*)a.x + (row < a.rows ? row : 0) * a.ldx;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * GT + lane) * V;
      raw[j] = load_pack<DT, V>(x + c, row < a.rows ? a.cols - c : 0);
    }
  };
  int64_t r0 = (int64_t)blockIdx.x * G;
  fetch(r0 + g);
  for (; r0 < a.rows; r0 += step) {
    const int64_t row = r0 + g;
    const bool live = row < a.rows;
    float v[NV][V];
    float s[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      unpack(raw[j], v[j]);
      s[0] += pair_sum(v[j]);
    }
    if constexpr (SAVE) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * GT + lane) * V;
        const int n = live ? a.cols - c : 0;
        Codes<V> q;
        const int sc = encode<DT, V>(raw[j], q);
        if (n > 0) {
          store_codes<V>(a.codes_out + row * a.cols + c, q, n);
          if (c % kBlock == 0)
            a.scales_out[row * ((a.cols + kBlock - 1) / kBlock) + c / kBlock] = (uint8_t)sc;
        }
      }
    }
    if (r0 + step < a.rows) fetch(row + step);
    row_sum<GT, 1>(s, lds, turn);
    const float mu = s[0] / n_f;
    s[0] = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int n = a.cols - (j * GT + lane) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[j][i] = i < n ? v[j][i] - mu : 0.0f;
        s[0] += v[j][i] * v[j][i];
      }
    }
    row_sum<GT, 1>(s, lds, turn);
    float mean = mu, var = s[0] / n_f;
    // the same in all lanes that meet at its barriers: a workgroup holds
    // several rows only where a row is a wave
    static_assert(G == 1 || GT == 64, "");
    if (row_far(mu, var, a.eps)) {
      s[0] = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) s[0] += pair_sum(v[j]);
      row_sum<GT, 1>(s, lds, turn);
      const float d = s[0] / n_f;
      row_correct(d, mean, var);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) v[j][i] -= d;
    }
    const float r = 1.0f / sqrtf(var + a.eps);
    if (!live) continue;
    E* const y = (E*)a.y + row * a.ldy;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * GT + lane) * V;
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = v[j][i] * r * w[j][i] + b[j][i];
      store_pack<DT, V>(y + c, pack<DT, V>(o), a.cols - c);
    }
    if (lane == 0 && a.mean) {
      a.mean[row] = mean;
      a.rstd[row] = r;
    }
  }
}

// x of a row's vector, from the matrix or the checkpoint
template <int DT, bool SAVED, int V>
struct Raw;
template <int DT, int V>
struct Raw<DT, false, V> {
  Pack<DT, V> q;
  __device__ __forceinline__ void load(const NormArgs& a, int64_t row, int c, int n) {
    q = load_pack<DT, V>((const elem_t<DT>*)a.x + row * a.ldx + c, n);
  }
  __device__ __forceinline__ void values(float (&v)[V]) const { unpack(q, v); }
};
template <int DT, int V>
struct Raw<DT, true, V> {
  Codes<V> q;
  int s;
  __device__ __forceinline__ void load(const NormArgs& a, int64_t row, int c, int n) {
    q = load_codes<V>(a.codes + row * a.cols + c, n);
    s = n > 0 ? a.scales[row * ((a.cols + kBlock - 1) / kBlock) + c / kBlock] : 0;
  }
  __device__ __forceinline__ void values(float (&v)[V]) const { decode<V>(q, s, v); }
};

// What the compiler knows of a value's registers ends here.
template <typename T>
__device__ __forceinline__ void hide(T& v) {
  static_assert(sizeof(T) % 4 == 0, "whole registers");
  uint32_t u[sizeof(T) / 4];
  __builtin_memcpy(u, &v, sizeof(T));
#pragma unroll
  for (uint32_t& x : u) asm volatile("" : "+v"(x));
  __builtin_memcpy(&v, u, sizeof(T));
}

// dx of every row, and the workgroup's partial sums of dw and db.
template <int DT, int PDT, int GT, int NV, int G, bool SAVED>
__global__ __launch_bounds__(GT* G) void norm_backward_kernel(NormArgs a) {
  constexpr int V = kVec<DT>;
  using E = elem_t<DT>;
  __shared__ float lds[2 * 16 * 2];
  const int lane = threadIdx.x % GT, g = threadIdx.x / GT;
  int turn = 0;
  float w[NV][V], dw[NV][V], db[NV][V];
  load_param<PDT, V, NV, GT>(a.weight, lane, a.cols, 1.0f, w);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) dw[j][i] = db[j][i] = 0.0f;
  const float n_f = (float)a.cols;
  const int64_t step = (int64_t)gridDim.x * G;

  // Two rows' loads: the one that is worked on and the next (a CU needs some
  // 30 KB under way to draw its share of memory's rate; a workgroup of 1024
  // lanes has 32 bytes of each lane's row).  To leave registers for them,
  // xh and h are made again from the loaded row after its sums have met,
  // not kept (55 us kept, 42 made again; a third row spills).
  constexpr int kAhead = 2;
  Raw<DT, SAVED, V> xr[kAhead][NV];
  Pack<DT, V> dr[kAhead][NV];
  float mu[kAhead], rs[kAhead];
  auto fetch = [&](int q, int64_t row) {
    const bool live = row < a.rows;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * GT + lane) * V;
      const int n = live ? a.cols - c : 0;
      xr[q][j].load(a, live ? row : 0, c, n);
      dr[q][j] = load_pack<DT, V>((const E*)a.dy + (live ? row : 0) * a.lddy + c, n);
    }
    mu[q] = live ? a.mean[row] : 0.0f;
    rs[q] = live ? a.rstd[row] : 0.0f;
  };
  auto work = [&](int q, int64_t row) {
    float s[2] = {0.0f, 0.0f};
    const float r = rs[q], m = mu[q];
    // xh, dy and h of vector j; a lane past the row's end has dy = 0, which
    // the sums take as it is, and xh must be 0, not -mu r (maybe NaN)
    auto values = [&](int j, float (&xh)[V], float (&d)[V], float (&h)[V]) {
      const int n = a.cols - (j * GT + lane) * V;
      xr[q][j].values(xh);
      unpack(dr[q][j], d);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        xh[i] = i < n ? (xh[i] - m) * r : 0.0f;
        h[i] = d[i] * w[j][i];
      }
    };
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float xh[V], d[V], h[V];
      values(j, xh, d, h);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[0] += h[i];
        s[1] += h[i] * xh[i];
        dw[j][i] += d[i] * xh[i];
        db[j][i] += d[i];
      }
    }
    row_sum<GT, 2>(s, lds, turn);
    if (row < a.rows && a.y) {
      const float m0 = s[0] / n_f, m1 = s[1] / n_f;
      E* const dx = (E*)a.y + row * a.ldy;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * GT + lane) * V;
        float xh[V], d[V], h[V], o[V];
        hide(xr[q][j]);
        hide(dr[q][j]);
        values(j, xh, d, h);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = r * (h[i] - m0 - xh[i] * m1);
        store_pack<DT, V>(dx + c, pack<DT, V>(o), a.cols - c);
      }
    }
    fetch(q, row + kAhead * step);
  };
  int64_t row = (int64_t)blockIdx.x * G + g;
#pragma unroll
  for (int q = 0; q < kAhead; ++q) fetch(q, row + q * step);
  // every group of the workgroup takes as many turns (rows past the end
  // are empty), for the barriers
  for (int64_t r0 = (int64_t)blockIdx.x * G; r0 < a.rows; r0 += kAhead * step) {
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      if (r0 + q * step >= a.rows) break;  // the whole workgroup
      work(q, row);
      row += step;
    }
  }
  if (!a.partial) return;
  // the G rows' sums meet in LDS, in group order, one vector a time
  float* const out = a.partial + (int64_t)blockIdx.x * 2 * a.cols;
  if constexpr (G == 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * GT + lane) * V;
      store_pack<kFP32, V>(out + c, pack<kFP32, V>(dw[j]), a.cols - c);
      store_pack<kFP32, V>(out + a.cols + c, pack<kFP32, V>(db[j]), a.cols - c);
    }
  } else {
    __shared__ float meet[G][GT * V];
#pragma unroll
    for (int k = 0; k < 2 * NV; ++k) {
      const int j = k >> 1;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < V; ++i) meet[g][i * GT + lane] = (k & 1) ? db[j][i] : dw[j][i];
      __syncthreads();
      for (int t = threadIdx.x; t < GT * V; t += GT * G) {
        const int c = j * GT * V + t;  // column, of lane t / V, element t % V
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < G; ++q) s += meet[q][(t % V) * GT + t / V];
        if (c < a.cols) out[(k & 1) * a.cols + c] = s;
      }
    }
  }
}

// Rows too long for registers: one workgroup a row, the row read again for
// each pass (from L2, as a row is at most a few hundred KB).
template <int DT, bool SAVE>
__global__ __launch_bounds__(1024) void norm_long_kernel(NormArgs a, int pdt) {
  constexpr int V = kVec<DT>, GT = 1024;
  using E = elem_t<DT>;
  __shared__ float lds[2 * 16];
  int turn = 0;
  const float n_f = (float)a.cols;
  // whole waves walk the row together, so that a block's lanes are all there
  const int end = (a.cols + 64 * V - 1) / (64 * V) * 64 * V;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const E* const x = (const E*)a.x + row * a.ldx;
    float s[1] = {0.0f};
    for (int c = threadIdx.x * V; c < end; c += GT * V) {
      const int n = a.cols - c;
      const Pack<DT, V> raw = load_pack<DT, V>(x + c, n);
      float v[V];
      unpack(raw, v);
      s[0] += pair_sum(v);
      if constexpr (SAVE) {
        Codes<V> q;
        const int sc = encode<DT, V>(raw, q);
        if (n > 0) {
          store_codes<V>(a.codes_out + row * a.cols + c, q, n);
          if (c % kBlock == 0)
            a.scales_out[row * ((a.cols + kBlock - 1) / kBlock) + c / kBlock] = (uint8_t)sc;
        }
      }
    }
    row_sum<GT, 1>(s, lds, turn);
    const float mu = s[0] / n_f;
    s[0] = 0.0f;
    for (int c = threadIdx.x * V; c < a.cols; c += GT * V) {
      float v[V];
      unpack(load_pack<DT, V>(x + c, a.cols - c), v);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c + i < a.cols) s[0] += (v[i] - mu) * (v[i] - mu);
    }
    row_sum<GT, 1>(s, lds, turn);
    float mean = mu, var = s[0] / n_f, d = 0.0f;
    if (row_far(mu, var, a.eps)) {
      s[0] = 0.0f;
      for (int c = threadIdx.x * V; c < a.cols; c += GT * V) {
        float v[V];
        unpack(load_pack<DT, V>(x + c, a.cols - c), v);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = c + i < a.cols ? v[i] - mu : 0.0f;
        s[0] += pair_sum(v);
      }
      row_sum<GT, 1>(s, lds, turn);
      d = s[0] / n_f;
      row_correct(d, mean, var);
    }
    const float r = 1.0f / sqrtf(var + a.eps);
    E* const y = (E*)a.y + row * a.ldy;
    for (int c = threadIdx.x * V; c < a.cols; c += GT * V) {
      float v[V];
      unpack(load_pack<DT, V>(x + c, a.cols - c), v);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c + i < a.cols) {
          const float w = a.weight ? load_any(a.weight, c + i, pdt) : 1.0f;
          const float b = a.bias ? load_any(a.bias, c + i, pdt) : 0.0f;
          v[i] = (v[i] - mu - d) * r * w + b;
        }
      store_pack<DT, V>(y + c, pack<DT, V>(v), a.cols - c);
    }
    if (threadIdx.x == 0 && a.mean) {
      a.mean[row] = mean;
      a.rstd[row] = r;
    }
  }
}

template <int DT, bool SAVED>
__global__ __launch_bounds__(1024) void norm_long_dx_kernel(NormArgs a, int pdt) {
  constexpr int V = kVec<DT>, GT = 1024;
  using E = elem_t<DT>;
  __shared__ float lds[2 * 16 * 2];
  int turn = 0;
  const float n_f = (float)a.cols;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float r = a.rstd[row], mu = a.mean[row];
    const E* const dy = (const E*)a.dy + row * a.lddy;
    E* const dx = (E*)a.y + row * a.ldy;
    float s[2] = {0.0f, 0.0f};
    float m0 = 0.0f, m1 = 0.0f;
    for (int pass = 0; pass < 2; ++pass) {
      for (int c = threadIdx.x * V; c < a.cols; c += GT * V) {
        const int n = a.cols - c;
        Raw<DT, SAVED, V> xr;
        float x[V], d[V];
        xr.load(a, row, c, n);
        xr.values(x);
        unpack(load_pack<DT, V>(dy + c, n), d);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (i >= n) break;
          const float w = a.weight ? load_any(a.weight, c + i, pdt) : 1.0f;
          const float xh = (x[i] - mu) * r, h = d[i] * w;
          if (pass == 0) {
            s[0] += h;
            s[1] += h * xh;
          } else {
            d[i] = r * (h - m0 - xh * m1);
          }
        }
        if (pass == 1) store_pack<DT, V>(dx + c, pack<DT, V>(d), n);
      }
      if (pass == 0) {
        row_sum<GT, 2>(s, lds, turn);
        m0 = s[0] / n_f;
        m1 = s[1] / n_f;
      }
    }
  }
}

// Partial sums of dw and db over a run of rows, for the columns of one
// workgroup (64 lanes of V columns each, four waves over the rows).
template <int DT, bool SAVED>
__global__ __launch_bounds__(256) void norm_long_dw_kernel(NormArgs a, int64_t run) {
  constexpr int V = kVec<DT>;
  using E = elem_t<DT>;
  __shared__ float meet[2][4][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = (blockIdx.x * 64 + lane) * V, n = a.cols - c;
  const int64_t r0 = blockIdx.y * run, r1 = r0 + run < a.rows ? r0 + run : a.rows;
  float dw[V], db[V];
#pragma unroll
  for (int i = 0; i < V; ++i) dw[i] = db[i] = 0.0f;
  if (n > 0)
    for (int64_t row = r0 + wave; row < r1; row += 4) {
      const float r = a.rstd[row], mu = a.mean[row];
      Raw<DT, SAVED, V> xr;
      float x[V], d[V];
      xr.load(a, row, c, n);
      xr.values(x);
      unpack(load_pack<DT, V>((const E*)a.dy + row * a.lddy + c, n), d);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        dw[i] += d[i] * ((x[i] - mu) * r);
        db[i] += d[i];
      }
    }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    meet[0][wave][i * 64 + lane] = dw[i];
    meet[1][wave][i * 64 + lane] = db[i];
  }
  __syncthreads();
  if (wave < 2) {
    float* const out = a.partial + ((int64_t)blockIdx.y * 2 + wave) * a.cols;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float s = 0.0f;
      for (int q = 0; q < 4; ++q) s += meet[wave][q][i * 64 + lane];
      if (i < n) out[c + i] = s;
    }
  }
}

// Column sums of `count` rows of partial sums, in row order within each of
// 16 runs and then in run order.  lane = column; blockIdx.y picks one of
// the interleaved matrices (row p of matrix y starts at (p * gridDim.y + y)
// * cols).
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* partial, int count,
                                                          int64_t cols, void* out0, void* out1,
                                                          int dt) {
  __shared__ float meet[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  void* const out = blockIdx.y ? out1 : out0;
  if (!out) return;  // the whole workgroup
  const int run = (count + 15) / 16;
  const int p0 = wave * run, p1 = p0 + run < count ? p0 + run : count;
  float s = 0.0f;
  if (c < cols) {
    const float* p = partial + blockIdx.y * cols + c;
    const int64_t stride = (int64_t)gridDim.y * cols;
#pragma unroll 16
    for (int q = p0; q < p1; ++q) s += p[q * stride];
  }
  meet[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < cols) {
    s = meet[0][lane];
#pragma unroll
    for (int w = 1; w < 16; ++w) s += meet[w][lane];
    store_any(out, c, s, dt);
  }
}

}  // namespace mmaops
#endif
