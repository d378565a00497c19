// saved.h -- 8-bit checkpoints of a matrix, their restoration, and the
// gradient of an activation with the bias's gradient.
//
// All of these read and write each element once and do little else, so
// memory bounds them: 16-byte loads, a wave's lanes along a row.  The 32
// elements of a checkpoint block sit in 4 neighbouring lanes (8 for FP32),
// whose largest magnitude takes two (three) exchanges.
//
// Measured: 8192 x 4096 bf16 (102 MB) saved in 20 us, restored in 16 us (from
// memory 19 and 18, 5.4 TB/s); the gradient of gelu with the bias's, 4096 x
// 4096 bf16 from a checkpoint (84 MB), in 27 us: its arithmetic, about 40
// instructions an element, takes longer than memory does (16 us).
#ifndef MMAOPS_SAVED_H
#define MMAOPS_SAVED_H

#include "norm.h"

namespace mmaops {

// A workgroup of 256 lanes is cut into rows of 2^shift lanes, as many as a
// row has vectors (16 at least, so that a block's lanes are always there).
template <int DT>
__global__ __launch_bounds__(256) void save_kernel(const void* x, int64_t ldx, uint8_t* codes,
                                                   uint8_t* scales, int64_t rows, int64_t cols,
                                                   int shift) {
  constexpr int V = kVec<DT>;
  const int lane = threadIdx.x & ((1 << shift) - 1), g = threadIdx.x >> shift;
  const int64_t step = (int64_t)gridDim.x * (256 >> shift);
  const int64_t nb = (cols + kBlock - 1) / kBlock, end = nb * kBlock;
  const int64_t c0 = ((int64_t)blockIdx.y << shift) * V, cstep = ((int64_t)gridDim.y << shift) * V;
  for (int64_t row = (int64_t)blockIdx.x * (256 >> shift) + g; row < rows; row += step)
    for (int64_t c = c0 + lane * V; c < end; c += cstep) {
      const int n = cols - c < V ? (int)(cols - c) : V;
      Codes<V> q;
      const int s =
          encode<DT, V>(load_pack<DT, V>((const elem_t<DT>*)x + row * ldx + c, n), q);
      if (n > 0) store_codes<V>(codes + row * cols + c, q, n);
      if (c % kBlock == 0) scales[row * nb + c / kBlock] = (uint8_t)s;
    }
}

template <int DT>
__global__ __launch_bounds__(256) void restore_kernel(const uint8_t* codes,
                                                      const uint8_t* scales, void* y,
                                                      int64_t ldy, int64_t rows, int64_t cols,
                                                      int shift) {
  constexpr int V = kVec<DT>;
  const int lane = threadIdx.x & ((1 << shift) - 1), g = threadIdx.x >> shift;
  const int64_t step = (int64_t)gridDim.x * (256 >> shift);
  const int64_t nb = (cols + kBlock - 1) / kBlock;
  const int64_t c0 = ((int64_t)blockIdx.y << shift) * V, cstep = ((int64_t)gridDim.y << shift) * V;
  for (int64_t row = (int64_t)blockIdx.x * (256 >> shift) + g; row < rows; row += step)
    for (int64_t c = c0 + lane * V; c < cols; c += cstep) {
      const int n = cols - c < V ? (int)(cols - c) : V;
      float v[V];
      decode<V>(load_codes<V>(codes + row * cols + c, n), scales[row * nb + c / kBlock], v);
      store_pack<DT, V>((elem_t<DT>*)y + row * ldy + c, pack<DT, V>(v), n);
    }
}

// A matrix of 16-bit elements copied to rows of ldy elements that start on
// 16 bytes, for the direct loads of a product.
__global__ __launch_bounds__(256) void align_kernel(const uint16_t* x, int64_t ldx, uint16_t* y,
                                                    int64_t ldy, int64_t rows, int64_t cols,
                                                    int shift) {
  constexpr int V = 8;
  const int lane = threadIdx.x & ((1 << shift) - 1), g = threadIdx.x >> shift;
  const int64_t step = (int64_t)gridDim.x * (256 >> shift);
  const int64_t c0 = ((int64_t)blockIdx.y << shift) * V, cstep = ((int64_t)gridDim.y << shift) * V;
  for (int64_t row = (int64_t)blockIdx.x * (256 >> shift) + g; row < rows; row += step)
    for (int64_t c = c0 + lane * V; c < cols; c += cstep) {
      const int n = cols - c < V ? (int)(cols - c) : V;
      store_pack<kBF16, V>((__bf16*)(y + row * ldy + c),
                           load_pack<kBF16, V>((const __bf16*)(x + row * ldx + c), n), V);
    }
}

struct DzArgs {
  const void* dy;
  int64_t lddy;
  const void* z;  // or codes and scales; neither with act none
  int64_t ldz;
  const uint8_t* codes;
  const uint8_t* scales;
  void* dz;  // rounded to the element type, row length N; NULL: not written
  int64_t lddz;
  float* partial;  // [gridDim.y][N] column sums before that rounding; NULL: none
  int64_t M, N;
  int64_t run;  // rows of one workgroup
  int act;
};

// dz = dy act'(z) and its column sums over the workgroup's run of rows: 64
// lanes of 8 columns, four waves over the rows, the waves' sums added in
// wave order.
template <int DT>
__global__ __launch_bounds__(256) void dz_kernel(DzArgs a) {
  constexpr int V = 8;
  using E = elem_t<DT>;
  __shared__ float meet[4][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = ((int64_t)blockIdx.x * 64 + lane) * V;
  const int n = a.N - c < V ? (int)(a.N - c) : V;
  const int64_t r0 = (int64_t)blockIdx.y * a.run, r1 = r0 + a.run < a.M ? r0 + a.run : a.M;
  const int64_t nb = (a.N + kBlock - 1) / kBlock;
  float db[V];
#pragma unroll
  for (int i = 0; i < V; ++i) db[i] = 0.0f;
  if (n > 0) {
    // kRows rows of the wave at once, so that their loads are all on their
    // way before the first is used
    constexpr int kRows = 2;
    for (int64_t row = r0 + wave; row < r1; row += 4 * kRows) {
      Pack<DT, V> dy[kRows], z[kRows];
      Codes<V> q[kRows];
      int sc[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int64_t m = row + 4 * u;
        const int k = m < r1 ? n : 0;
        dy[u] = load_pack<DT, V>((const E*)a.dy + m * a.lddy + c, k);
        if (a.act == kActNone) continue;
        if (a.codes) {
          q[u] = load_codes<V>(a.codes + m * a.N + c, k);
          sc[u] = k ? a.scales[m * nb + c / kBlock] : 0;
        } else {
          z[u] = load_pack<DT, V>((const E*)a.z + m * a.ldz + c, k);
        }
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int64_t m = row + 4 * u;
        float d[V];
        unpack(dy[u], d);
        if (a.act != kActNone) {
          float t[V];
          if (a.codes)
            decode<V>(q[u], sc[u], t);
          else
            unpack(z[u], t);
          act_all(t, a.act, act_slope);
#pragma unroll
          for (int i = 0; i < V; ++i) d[i] *= t[i];
        }
        if (m >= r1) continue;
        if (a.dz) store_pack<DT, V>((E*)a.dz + m * a.lddz + c, pack<DT, V>(d), n);
#pragma unroll
        for (int i = 0; i < V; ++i) db[i] += d[i];
      }
    }
  }
  if (!a.partial) return;
#pragma unroll
  for (int i = 0; i < V; ++i) meet[wave][i * 64 + lane] = db[i];
  __syncthreads();
  float* const out = a.partial + (int64_t)blockIdx.y * a.N;
  for (int t = threadIdx.x; t < 64 * V; t += 256) {
    const int64_t col = (int64_t)blockIdx.x * 64 * V + t;
    const int at = (t % V) * 64 + t / V;
    if (col < a.N) out[col] = meet[0][at] + meet[1][at] + meet[2][at] + meet[3][at];
  }
}

}  // namespace mmaops
#endif
