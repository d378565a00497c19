// gated.h -- a gated layer, Y = act(X Wg + bg) (X Wu + bu), and its backward
// pass, on the products of linear.h.
//
// Forward.  Both weights are right operands of one product: a tile holds the
// same columns of both, so that a wave has their sums in the same lanes and the
// epilogue multiplies them where they are; neither goes through memory unless
// it is to be kept.
//
// Backward.  One pass over dY and what was kept gives
//   dg = dY u act'(g),  du = dY act(g)
// rounded to the operands' type, which is what the matrix cores multiply at their rate
// (as dz of a plain product: in FP16 past 65504 an infinity, as in any 16-bit gradient),
// and their column sums before that.  Then
//   dX = dg Wg^T + du Wu^T   one product with an inner size of 2 N
//   dWg = X^T dg, dWu = X^T du   the tiles of both in one launch
//
// Measured (one MI355X).  4096 x 4096 x 4096 bf16, gelu, both biases: 207 us and more for
// 275 GFLOP (1.33 PFLOP/s, the plain product's rate; 569 on small tiles).  Its
// backward pass from checkpoints: dg and du 33 (silu 29), dX 210 (both W N x K 229), both
// dW 240.  1 x 4096 x 4096 bf16, both W N x K: 13 (67 MB, again and again; 16 from
// memory, 4.2 TB/s).
#ifndef MMAOPS_GATED_H
#define MMAOPS_GATED_H

#include "linear.h"

namespace mmaops {

template <int DT, int BM, int BN, int BK, int WM, int WN, int LB, int STAGES, bool DIRECT,
          int MODE>
__global__ __launch_bounds__(WM* WN * 64, 2) void joint_kernel(args_t<MODE> g) {
  __shared__ __attribute__((aligned(1024))) char smem[kRingBytes<BM, BN, BK, STAGES>];
  const int block = (int)(blockIdx.x + blockIdx.z * (uint32_t)g.grid_x);
  if (block >= g.tiles_m * g.tiles_n) return;  // the whole workgroup
  small_product<DT, BM, BN, BK, WM, WN, 0, LB, STAGES, DIRECT, MODE>(g, block, blockIdx.y, smem);
}

template <int DT, int BM, int BN, int LB, int STAGES, int MODE>
__global__ __launch_bounds__(256, 1) void joint_wide_kernel(args_t<MODE> g) {
  __shared__ __attribute__((aligned(1024))) char smem[Wide<BM, BN, STAGES>::kBytes];
  const int block = (int)(blockIdx.x + blockIdx.z * (uint32_t)g.grid_x);
  if (block >= g.tiles_m * g.tiles_n) return;  // the whole workgroup
  wide_product<DT, 0, LB, BM, BN, STAGES, MODE>(g, block, blockIdx.y, smem);
}

// Up to 16 rows in one launch, BN / 2 output columns a workgroup: bound by the
// weights' bytes.
template <int DT, int LB, int BN>
__global__ __launch_bounds__(512, 2) void gate_rows_kernel(GateArgs g) {
  __shared__ __attribute__((aligned(1024))) char smem[kRowsBytes];
  rows_product<DT, LB, BN, kGate>(g, smem);
}

// Two products of the same sizes and layouts, one's tiles after the other's.
struct TwoArgs {
  LinearArgs one, two;
};

template <int DT, int BM, int BN, int STAGES>
__global__ __launch_bounds__(256, 1) void two_wide_kernel(TwoArgs p) {
  __shared__ __attribute__((aligned(1024))) char smem[Wide<BM, BN, STAGES>::kBytes];
  const int n = p.one.tiles_m * p.one.tiles_n;
  const int64_t block = blockIdx.x + (int64_t)blockIdx.z * p.one.grid_x;
  if (block >= 2 * (int64_t)n) return;  // the whole workgroup
  wide_product<DT, 1, 1, BM, BN, STAGES, kPlain>(
      block < n ? p.one : p.two, (int)(block < n ? block : block - n), blockIdx.y, smem);
}

template <int DT, int BM, int BN, int BK, int WM, int WN, int STAGES, bool DIRECT>
__global__ __launch_bounds__(WM* WN * 64, 2) void two_kernel(TwoArgs p) {
  __shared__ __attribute__((aligned(1024))) char smem[kRingBytes<BM, BN, BK, STAGES>];
  const int n = p.one.tiles_m * p.one.tiles_n;
  const int64_t block = blockIdx.x + (int64_t)blockIdx.z * p.one.grid_x;
  if (block >= 2 * (int64_t)n) return;  // the whole workgroup
  small_product<DT, BM, BN, BK, WM, WN, 1, 1, STAGES, DIRECT>(
      block < n ? p.one : p.two, (int)(block < n ? block : block - n), blockIdx.y, smem);
}

// A small backward pass's second launch: the tiles of dg Wg^T + du Wu^T, those of
// both weight gradients, then the column sums of both biases, 64 columns a
// workgroup; all need only the first launch's results.  Launches bound such a
// pass (fp16, gelu, 299 x 260 x 640, on the GPU: four launches 27 us, two 14.5).
struct SmallArgs {
  LongArgs dx;
  TwoArgs dw;
  const float* partial;  // [count][2][cols]
  void *dbias_g, *dbias_u;
  int64_t cols;
  int count, dbias_dt;  // count 0: no sums
};

template <int DT, int LB>
__global__ __launch_bounds__(256, 2) void gated_small_kernel(SmallArgs p) {
  __shared__ __attribute__((aligned(1024))) char smem[kRingBytes<64, 64, 64, 3>];
  const int n1 = p.dx.tiles_m * p.dx.tiles_n, n2 = p.dw.one.tiles_m * p.dw.one.tiles_n;
  const int b = blockIdx.x;
  if (b < n1) {
    small_product<DT, 64, 64, 64, 2, 2, 0, LB, 3, true, kLong>(p.dx, b, 0, smem);
  } else if (b < n1 + 2 * n2) {
    const int t = b - n1;
    small_product<DT, 64, 64, 64, 2, 2, 1, 1, 3, true>(t < n2 ? p.dw.one : p.dw.two,
                                                       t < n2 ? t : t - n2, 0, smem);
  } else {
    // in the runs and the order of column_sum_kernel, for the same bits
    float(&meet)[16][64] = *(float(*)[16][64])smem;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int blocks = (int)((p.cols + 63) / 64), t = b - n1 - 2 * n2;
    const int which = t < blocks ? 0 : 1;
    void* const out = which ? p.dbias_u : p.dbias_g;
    const int64_t c = (int64_t)(t - which * blocks) * 64 + lane;
    const int run = (p.count + 15) / 16;
    // four of the sixteen runs a wave, side by side; past a run's end + 0
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < p.cols) {
#pragma unroll 4
      for (int q = 0; q < run; ++q) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = (wave * 4 + i) * run + q;
          s[i] += row < p.count ? p.partial[((int64_t)row * 2 + which) * p.cols + c] : 0.0f;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) meet[wave * 4 + i][lane] = s[i];
    __syncthreads();
    if (wave == 0 && c < p.cols && out) {
      float sum = meet[0][lane];
#pragma unroll
      for (int r = 1; r < 16; ++r) sum += meet[r][lane];
      store_any(out, c, sum, p.dbias_dt);
    }
  }
}

// The runs' sums of both halves added in run order, then the epilogue: four
// columns a lane, eight neighbouring lanes for a checkpoint block.  A launch's
// fixed cost, mostly (16 x 8192: 4.2 to 4.7 us for two runs or four).
template <int DT>
__global__ __launch_bounds__(64) void gate_finish_kernel(GateArgs g) {
  const int64_t quads = (g.N + kBlock - 1) / kBlock * (kBlock / 4);  // of a row
  const int64_t total = quads * g.M;
  for (int64_t t = (int64_t)blockIdx.x * 64 + threadIdx.x; t < total;
       t += (int64_t)gridDim.x * 64) {
    const int64_t m = t / quads, c = (t - m * quads) * 4;
    const int n = g.N - c < 4 ? (int)(g.N - c) : 4;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f}, u[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (n > 0) {
      // four runs' sums of both on their way at once
      const float* p = g.partial + m * 2 * g.N + c;
      const int64_t run = g.M * 2 * g.N;
      for (int s0 = 0; s0 < g.splits; s0 += 4) {
        Pack<kFP32, 4> a[4], b[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int k = s0 + s < g.splits ? n : 0;
          a[s] = load_pack<kFP32, 4>(p + (s0 + s) * run, k);
          b[s] = load_pack<kFP32, 4>(p + (s0 + s) * run + g.N, k);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          float w[4], z[4];
          unpack(a[s], w);
          unpack(b[s], z);
          if (s0 + s < g.splits) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v[i] = s0 + s ? v[i] + w[i] : w[i];
              u[i] = s0 + s ? u[i] + z[i] : z[i];
            }
          }
        }
      }
      float bias[4], bias2[4];
      gate_bias<4>(g, c, n, bias, bias2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] += bias[i];
        u[i] += bias2[i];
      }
    }
    if (g.codes) gate_save<DT, 4>(g, m, c, n, v, u);  // a block's lanes are here together
    gate_finish<DT, 4, 1>(g, m, 0, c, n, false, v, u);
  }
}

// ------------------------------------------------------------ backward
struct GateDzArgs {
  const void* dy;
  int64_t lddy;
  const void *g, *u;  // or codes and scales of both
  int64_t ldg, ldu;
  const uint8_t *g_codes, *g_scales, *u_codes, *u_scales;
  void *dg, *du;  // row length N, NULL: not written
  int64_t ldd;
  float* partial;  // [gridDim.y][2][N] column sums of dg and du, NULL: none
  int64_t M, N;
  int64_t run;  // rows of one workgroup
  int act;
};

// What was kept whole may be an infinity where the forward pass had a number,
// past its 16 bits: taken as a number, a gate far below 0 gives 0 (and not 0
// times infinity).  That number is the largest of BF16, for FP16 one past its own:
// finite values stay, and so does NaN.
template <int DT>
__device__ __forceinline__ void as_numbers(float (&v)[8]) {
  constexpr float kFar = DT == kFP16 ? 1e30f : 0x1.FEp127f;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = v[i] > kFar ? kFar : v[i] < -kFar ? -kFar : v[i];
}

// act(z) and its slope of V values, as act_apply and act_slope have them, what
// both need made once (gelu's tail, a logistic).
template <int V>
__device__ __forceinline__ void act_both(const float (&z)[V], const int act, float (&f)[V],
                                         float (&s)[V]) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int i = 0; i < V; ++i) {
        f[i] = z[i] < 0.0f ? 0.0f : z[i];
        s[i] = z[i] > 0.0f ? 1.0f : 0.0f;
      }
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float b = bounded(z[i], kTailEnd), a = __builtin_fabsf(b), q = normal_tail(a);
        const float e = fast_exp2(z[i] * z[i] * (-0.5f * kLog2e));
        f[i] = __builtin_fmaf(-a, q, z[i] < 0.0f ? 0.0f : z[i]);
        s[i] = __builtin_fmaf(b * e, kInvSqrt2Pi, z[i] > 0.0f ? 1.0f - q : q);
      }
      break;
    case kActGeluTanh:
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float b = z[i] > 12.0f ? 12.0f : z[i] < -12.0f ? -12.0f : z[i], b2 = b * b;
        const float l = logistic(2.0f * kSqrt2OverPi * b * __builtin_fmaf(0.044715f, b2, 1.0f));
        f[i] = z[i] * l;
        s[i] = l + b * l * (1.0f - l) * 2.0f * kSqrt2OverPi * (1.0f + 3.0f * 0.044715f * b2);
      }
      break;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float l = logistic(z[i]);
        f[i] = z[i] * l;
        s[i] = l * (1.0f + bounded(z[i], 100.0f) * (1.0f - l));
      }
      break;
    default:
#pragma unroll
      for (int i = 0; i < V; ++i) {
        f[i] = z[i];
        s[i] = 1.0f;
      }
  }
}

// dg, du and their column sums over the workgroup's run of rows: 64 lanes of
// 8 columns, four waves over the rows, the waves' sums added in wave order.  The
// activation is the kernel's own: with a switch in it, it held the registers
// of the largest.  Bound by memory (4096 x 4096 bf16 from both checkpoints: silu 26.3
// to 28.6 us for 135 MB, 5 TB/s; gelu's arithmetic 30 to 35), so dg and du leave in one
// pass.
template <int DT, int ACT, bool SAVED>
__global__ __launch_bounds__(256, 4) void gate_dz_kernel(GateDzArgs a) {
  constexpr int V = 8;
  using E = elem_t<DT>;
  __shared__ float meet[4][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = ((int64_t)blockIdx.x * 64 + lane) * V;
  const int n = a.N - c < V ? (int)(a.N - c) : V;
  const int64_t r0 = (int64_t)blockIdx.y * a.run, r1 = r0 + a.run < a.M ? r0 + a.run : a.M;
  const int64_t nb = (a.N + kBlock - 1) / kBlock;
  float sg[V], su[V];
#pragma unroll
  for (int i = 0; i < V; ++i) sg[i] = su[i] = 0.0f;
  if (n > 0) {
    for (int64_t m = r0 + wave; m < r1; m += 4) {
      float d[V], g[V], u[V];
      const Pack<DT, V> py = load_pack<DT, V>((const E*)a.dy + m * a.lddy + c, n);
      if constexpr (SAVED) {
        const int64_t at = m * nb + c / kBlock;
        const Codes<V> qg = load_codes<V>(a.g_codes + m * a.N + c, n);
        const Codes<V> qu = load_codes<V>(a.u_codes + m * a.N + c, n);
        const int eg = a.g_scales[at], eu = a.u_scales[at];
        decode<V>(qg, eg, g);
        decode<V>(qu, eu, u);
      } else {
        const Pack<DT, V> pg = load_pack<DT, V>((const E*)a.g + m * a.ldg + c, n);
        const Pack<DT, V> pu = load_pack<DT, V>((const E*)a.u + m * a.ldu + c, n);
        unpack(pg, g);
        unpack(pu, u);
        as_numbers<DT>(g);
        as_numbers<DT>(u);
      }
      unpack(py, d);
      float f[V], s[V];
      act_both<V>(g, ACT, f, s);
      // u may be as large as a float can be, and the slope 1.13: half of their
      // product is a number, which a dy of 0 makes 0.  Powers of two move no other
      // bits (above the subnormal numbers).
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float dg = d[i] * (u[i] * (0.5f * s[i])) * 2.0f, du = d[i] * f[i];
        g[i] = i < n ? dg : 0.0f;
        u[i] = i < n ? du : 0.0f;
        sg[i] += g[i];
        su[i] += u[i];
      }
      if (a.dg) {
        store_pack<DT, V>((E*)a.dg + m * a.ldd + c, pack<DT, V>(g), n);
        store_pack<DT, V>((E*)a.du + m * a.ldd + c, pack<DT, V>(u), n);
      }
    }
  }
  if (!a.partial) return;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (k) __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) meet[wave][i * 64 + lane] = k ? su[i] : sg[i];
    __syncthreads();
    float* const out = a.partial + ((int64_t)blockIdx.y * 2 + k) * a.N;
    for (int t = threadIdx.x; t < 64 * V; t += 256) {
      const int64_t col = (int64_t)blockIdx.x * 64 * V + t;
      const int at = (t % V) * 64 + t / V;
      if (col < a.N) out[col] = meet[0][at] + meet[1][at] + meet[2][at] + meet[3][at];
    }
  }
}

// ------------------------------------------------------------ variants
// a grid has fewer than 2^32 lanes in x
constexpr uint32_t kMostBlocks = 1u << 23;

inline dim3 joint_grid(int64_t blocks, int splits, int& grid_x) {
  grid_x = (int)(blocks < kMostBlocks ? blocks : kMostBlocks);
  return dim3((uint32_t)grid_x, (uint32_t)splits,
              (uint32_t)((blocks + kMostBlocks - 1) / kMostBlocks));
}

template <int DT, int LB>
hipError_t gate_launch_tile(int tile, bool direct, GateArgs g, hipStream_t s) {
  if (tile == kTileRows) {
    if (g.codes)
      gate_rows_kernel<DT, LB, 64><<<dim3((uint32_t)((g.N + 31) / 32)), 512, 0, s>>>(g);
    else
      gate_rows_kernel<DT, LB, 32><<<dim3((uint32_t)((g.N + 15) / 16)), 512, 0, s>>>(g);
    return hipGetLastError();
  }
  const dim3 grid = joint_grid((int64_t)g.tiles_m * g.tiles_n, g.splits, g.grid_x);
  // 128 x 128: three stages for one workgroup a CU, as in linear_launch_tile
  const bool alone = (int64_t)grid.x * grid.y * grid.z <= kCUs;
  if (tile == kTileBig)
    joint_wide_kernel<DT, 256, 256, LB, 2, kGate><<<grid, 256, 0, s>>>(g);
  else if (tile == kTileMid && alone)
    joint_wide_kernel<DT, 128, 128, LB, 3, kGate><<<grid, 256, 0, s>>>(g);
  else if (tile == kTileMid)
    joint_wide_kernel<DT, 128, 128, LB, 2, kGate><<<grid, 256, 0, s>>>(g);
  else if (tile == kTileSmall)
    joint_kernel<DT, 64, 64, 64, 2, 2, LB, 3, true, kGate><<<grid, 256, 0, s>>>(g);
  else if (direct)
    joint_kernel<DT, 16, 128, 128, 1, 4, LB, 3, true, kGate><<<grid, 256, 0, s>>>(g);
  else
    joint_kernel<DT, 16, 128, 128, 1, 4, LB, 2, false, kGate><<<grid, 256, 0, s>>>(g);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !g.partial) return e;
  const int64_t lanes = (g.N + kBlock - 1) / kBlock * (kBlock / 4) * g.M;
  const int64_t blocks = (lanes + 63) / 64;
  gate_finish_kernel<DT><<<(uint32_t)(blocks < 65536 ? blocks : 65536), 64, 0, s>>>(g);
  return hipGetLastError();
}

template <int DT>
hipError_t finish_launch(const LinearArgs& g, hipStream_t s) {
  const int64_t lanes = (g.N + kBlock - 1) / kBlock * (kBlock / 4) * g.M;
  const int64_t blocks = (lanes + 63) / 64;
  linear_finish_kernel<DT><<<(uint32_t)(blocks < 65536 ? blocks : 65536), 64, 0, s>>>(g);
  return hipGetLastError();
}

template <int DT, int LB>
hipError_t long_launch_tile(int tile, bool direct, LongArgs g, hipStream_t s) {
  const dim3 grid = joint_grid((int64_t)g.tiles_m * g.tiles_n, g.splits, g.grid_x);
  // 128 x 128: three stages for one workgroup a CU, as in linear_launch_tile
  const bool alone = (int64_t)grid.x * grid.y * grid.z <= kCUs;
  if (tile == kTileBig)
    joint_wide_kernel<DT, 256, 256, LB, 2, kLong><<<grid, 256, 0, s>>>(g);
  else if (tile == kTileMid && alone)
    joint_wide_kernel<DT, 128, 128, LB, 3, kLong><<<grid, 256, 0, s>>>(g);
  else if (tile == kTileMid)
    joint_wide_kernel<DT, 128, 128, LB, 2, kLong><<<grid, 256, 0, s>>>(g);
  else if (tile == kTileSmall)
    joint_kernel<DT, 64, 64, 64, 2, 2, LB, 3, true, kLong><<<grid, 256, 0, s>>>(g);
  else if (direct)
    joint_kernel<DT, 16, 64, 128, 1, 4, LB, 3, true, kLong><<<grid, 256, 0, s>>>(g);
  else
    joint_kernel<DT, 16, 64, 128, 1, 4, LB, 2, false, kLong><<<grid, 256, 0, s>>>(g);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess || !g.partial ? e : finish_launch<DT>(g, s);
}

template <int DT>
hipError_t two_launch(int tile, bool direct, TwoArgs p, hipStream_t s) {
  const dim3 grid =
      joint_grid(2 * (int64_t)p.one.tiles_m * p.one.tiles_n, p.one.splits, p.one.grid_x);
  const bool alone = (int64_t)grid.x * grid.y * grid.z <= kCUs;
  if (tile == kTileBig)
    two_wide_kernel<DT, 256, 256, 2><<<grid, 256, 0, s>>>(p);
  else if (tile == kTileMid && alone)
    two_wide_kernel<DT, 128, 128, 3><<<grid, 256, 0, s>>>(p);
  else if (tile == kTileMid)
    two_wide_kernel<DT, 128, 128, 2><<<grid, 256, 0, s>>>(p);
  else if (tile == kTileSmall)
    two_kernel<DT, 64, 64, 64, 2, 2, 3, true><<<grid, 256, 0, s>>>(p);
  else if (direct)
    two_kernel<DT, 16, 64, 128, 1, 4, 3, true><<<grid, 256, 0, s>>>(p);
  else
    two_kernel<DT, 16, 64, 128, 1, 4, 2, false><<<grid, 256, 0, s>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !p.one.partial) return e;
  e = finish_launch<DT>(p.one, s);
  return e != hipSuccess ? e : finish_launch<DT>(p.two, s);
}

template <int DT>
hipError_t gate_dz_launch(const GateDzArgs& d, int64_t runs, hipStream_t s) {
  const dim3 grid((uint32_t)((d.N + 511) / 512), (uint32_t)runs);
  const auto go = [&](auto act) {
    constexpr int ACT = decltype(act)::value;
    if (d.g_codes)
      gate_dz_kernel<DT, ACT, true><<<grid, 256, 0, s>>>(d);
    else
      gate_dz_kernel<DT, ACT, false><<<grid, 256, 0, s>>>(d);
  };
  switch (d.act) {
    case kActRelu: go(std::integral_constant<int, kActRelu>{}); break;
    case kActGelu: go(std::integral_constant<int, kActGelu>{}); break;
    case kActGeluTanh: go(std::integral_constant<int, kActGeluTanh>{}); break;
    case kActSilu: go(std::integral_constant<int, kActSilu>{}); break;
    default: go(std::integral_constant<int, kActNone>{});
  }
  return hipGetLastError();
}

// The launches of one element type; lb: the layout of the right operand.
struct GatedLaunches {
  hipError_t (*gate)(int tile, bool direct, int lb, const GateArgs& g, hipStream_t s);
  hipError_t (*both)(int tile, bool direct, int lb, const LongArgs& g, hipStream_t s);
  hipError_t (*two)(int tile, bool direct, const TwoArgs& p, hipStream_t s);
  hipError_t (*dz)(const GateDzArgs& d, int64_t runs, hipStream_t s);
  hipError_t (*small)(int lb, const SmallArgs& p, hipStream_t s);
};

template <int DT>
GatedLaunches gated_launches() {
  return {[](int tile, bool direct, int lb, const GateArgs& g, hipStream_t s) {
            return lb ? gate_launch_tile<DT, 1>(tile, direct, g, s)
                      : gate_launch_tile<DT, 0>(tile, direct, g, s);
          },
          [](int tile, bool direct, int lb, const LongArgs& g, hipStream_t s) {
            return lb ? long_launch_tile<DT, 1>(tile, direct, g, s)
                      : long_launch_tile<DT, 0>(tile, direct, g, s);
          },
          [](int tile, bool direct, const TwoArgs& p, hipStream_t s) {
            return two_launch<DT>(tile, direct, p, s);
          },
          [](const GateDzArgs& d, int64_t runs, hipStream_t s) {
            return gate_dz_launch<DT>(d, runs, s);
          },
          [](int lb, const SmallArgs& p, hipStream_t s) {
            const int64_t sums = p.count ? 2 * ((p.cols + 63) / 64) : 0;
            const uint32_t grid =
                (uint32_t)((int64_t)p.dx.tiles_m * p.dx.tiles_n +
                           2 * (int64_t)p.dw.one.tiles_m * p.dw.one.tiles_n + sums);
            if (lb)
              gated_small_kernel<DT, 1><<<grid, 256, 0, s>>>(p);
            else
              gated_small_kernel<DT, 0><<<grid, 256, 0, s>>>(p);
            return hipGetLastError();
          }};
}

GatedLaunches gated_fp16();
GatedLaunches gated_bf16();

}  // namespace mmaops
#endif
