// linear.h -- the matrix products of a layer and its backward pass on the
// matrix cores: C = A B with FP16 or BF16 operands, FP32 sums, and an
// epilogue that adds the bias, saves the pre-activation (whole or as a
// checkpoint), applies the activation and adds the residual before the one
// rounding of the output.
//
// Layout.  An operand is stored with its K index running fastest (layout
// 0) or with its row (A) or column (B) index running fastest (layout 1).
// The three products of a layer are then one kernel:
//   X W     A = X   layout 0, B = W   layout 1 (W stored K x N) or 0 (N x K)
//   dz W^T  A = dz  layout 0, B = W^T layout 0 or 1
//   X^T dz  A = X^T layout 1, B = dz  layout 1
// A tile goes to LDS as it is stored, by direct global->LDS loads of 16
// bytes a lane; layout 1 is turned on the way to the registers by the
// transposing LDS read, so that no operand is ever rearranged in memory.
//
// LDS banks.  A layout-0 tile row is BK elements; 16-byte chunk c of row r
// is kept at chunk c ^ (r & 7), so that the 16 rows of a fragment read
// spread over the banks.  A layout-1 tile row is one k with R columns;
// 32-byte slot s of row k is kept at s ^ g(k), with g taking 8 values over
// the 8 rows that half a wave reads at once.  The permutation is applied
// to the global address of each lane, as the LDS side of a direct load is
// always lane after lane.
//
// The matrix instruction takes B's fragment first: each lane then holds
// four neighbouring columns of one row of C.
#ifndef MMAOPS_LINEAR_H
#define MMAOPS_LINEAR_H

#include "ops_common.h"

namespace mmaops {

struct LinearArgs {
  const void* a;
  const void* b;
  int64_t lda, ldb;  // elements
  int64_t M, N, K;
  // splits > 1, or partial != NULL: the FP32 sums of each run of K go to
  // partial[split][M][N] and linear_finish_kernel does the rest
  int splits;
  int tiles_m, tiles_n;
  float* partial;
  // epilogue
  const void* bias;
  const void* residual;
  void* y;
  void* z;
  uint8_t* codes;
  uint8_t* scales;
  int64_t ldr, ldy, ldz;
  int bias_dt, out_dt, act;
};

template <int DT>
struct Mfma;
template <>
struct Mfma<kFP16> {
  using frag = half8;
  static __device__ __forceinline__ f32x4 run(frag a, frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Mfma<kBF16> {
  using frag = bf8;
  static __device__ __forceinline__ f32x4 run(frag a, frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};

using lds_char = __attribute__((address_space(3))) char;

// 16 bytes a lane from base + off to LDS at lds + 16 * lane (lds and base
// wave-uniform).  Written out so that the compiler does not wait for it
// before every LDS read; the waits are explicit.  It writes no register.
__device__ __forceinline__ void load_to_lds(const char* base, uint32_t off, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %2\n\t"
      "global_load_lds_dwordx4 %0, %1"
      :
      : "v"(off), "s"(base), "s"(lds)
      : "memory", "m0");
}

template <int N>
__device__ __forceinline__ void wait_loads() {  // all but the last N, and all LDS reads
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(N) : "memory");
}

// One operand's tile: R rows (or columns) by BK, NW waves loading it.
template <int R, int BK, int LAYOUT, int NW>
struct Tile {
  static constexpr int kBytes = R * BK * 2;
  static constexpr int kLoads = R * BK / 512;     // wave loads of 1 KiB
  static constexpr int kPerWave = kLoads / NW;
  static_assert(kLoads % NW == 0, "every wave issues the same number of loads");
  static constexpr int kRow = LAYOUT == 0 ? BK / 8 : R / 8;  // chunks of a tile row

  static __device__ __forceinline__ int swap_of(int r) {
    if constexpr (LAYOUT == 0) return r & (kRow < 8 ? kRow - 1 : 7);
    constexpr int slots = R / 16;
    return ((r & 3) | ((r >> 3) & 1) << 2) & (slots < 8 ? slots - 1 : 7);
  }
  // tile row, and the chunk of it that is kept at LDS chunk q
  static __device__ __forceinline__ void place(int q, int& row, int& chunk) {
    row = q / kRow;
    const int p = q % kRow;
    if constexpr (LAYOUT == 0)
      chunk = p ^ swap_of(row);
    else
      chunk = ((p >> 1) ^ swap_of(row)) * 2 + (p & 1);
  }

  // byte offsets of the lane's chunks from the tile's first element; rows
  // past the matrix (`have` rows are there) repeat the last one: what they
  // give is never stored
  static __device__ __forceinline__ void offsets(int64_t ld, int have, int wave, int lane,
                                                 uint32_t (&off)[kPerWave]) {
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) {
      int row, chunk;
      place((wave * kPerWave + i) * 64 + lane, row, chunk);
      if constexpr (LAYOUT == 0)
        row = row < have ? row : have - 1;
      else
        chunk = chunk * 8 < have ? chunk : have / 8 - 1;
      off[i] = (uint32_t)(row * ld * 2) + chunk * 16;
    }
  }
  static __device__ __forceinline__ void load(const char* base, const uint32_t (&off)[kPerWave],
                                              uint32_t lds, int wave) {
#pragma unroll
    for (int i = 0; i < kPerWave; ++i)
      load_to_lds(base, off[i], lds + (wave * kPerWave + i) * 1024);
  }

  // The same through registers, for any alignment and for a tile with only
  // `kn` of its BK (the rest 0): `have` rows, element by element where a
  // chunk passes an edge.
  static __device__ __forceinline__ void fetch(const char* tile, int64_t ld, int have, int kn,
                                               int wave, int lane, u32x4 (&v)[kPerWave]) {
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) {
      int row, chunk;
      place((wave * kPerWave + i) * 64 + lane, row, chunk);
      const int rows = LAYOUT == 0 ? have : kn, cols = LAYOUT == 0 ? kn : have;
      const char* p = tile + ((int64_t)row * ld + chunk * 8) * 2;
      v[i] = u32x4{0, 0, 0, 0};
      if (row < rows) {
        const int n = cols - chunk * 8;
        if (n >= 8) {
          __builtin_memcpy(&v[i], p, 16);
        } else {
          const uint16_t* e = (const uint16_t*)p;
#pragma unroll
          for (int j = 0; j < 7; ++j)
            if (j < n) v[i][j >> 1] |= (uint32_t)e[j] << (16 * (j & 1));
        }
      }
    }
  }
  static __device__ __forceinline__ void put(lds_char* tile, int wave, int lane,
                                             const u32x4 (&v)[kPerWave]) {
#pragma unroll
    for (int i = 0; i < kPerWave; ++i)
      *(__attribute__((address_space(3))) u32x4*)(tile + (wave * kPerWave + i) * 1024 +
                                                  lane * 16) = v[i];
  }

  // fragment of rows r0 .. r0 + 15 for k in [32 kk, 32 kk + 32): the lane
  // has row r0 + (lane & 15) and 8 k from 8 (lane >> 4)
  template <typename F>
  static __device__ __forceinline__ F frag(const lds_char* tile, int r0, int kk, int lane) {
    if constexpr (LAYOUT == 0) {
      const int row = r0 + (lane & 15), c = kk * 4 + (lane >> 4);
      return *(const __attribute__((address_space(3))) F*)(tile + row * (BK * 2) +
                                                           ((c ^ swap_of(row)) * 16));
    } else {
      using s4 = __attribute__((ext_vector_type(4))) short;
      union {
        s4 h[2];
        F f;
      } u;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = kk * 32 + (lane >> 4) * 8 + h * 4 + ((lane & 15) >> 2);
        u.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s4*)(tile + k * (R * 2) +
                                                    (((r0 / 16) ^ swap_of(k)) * 32) +
                                                    (lane & 3) * 8));
      }
      return u.f;
    }
  }
};

// ------------------------------------------------------------ epilogue
// Bias, pre-activation, activation, residual and store of four columns of
// one row; n of them are there.
template <int DT>
__device__ __forceinline__ void finish4(const LinearArgs& g, int64_t m, int64_t c, int n,
                                        float (&v)[4]) {
  using E = elem_t<DT>;
  if (g.z) store_pack<DT, 4>((E*)g.z + m * g.ldz + c, pack<DT, 4>(v), n);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = act_apply(v[i], g.act);
  if (g.out_dt == kFP32) {
    if (g.residual) {
      float r[4];
      unpack(load_pack<kFP32, 4>((const float*)g.residual + m * g.ldr + c, n), r);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += r[i];
    }
    store_pack<kFP32, 4>((float*)g.y + m * g.ldy + c, pack<kFP32, 4>(v), n);
  } else {
    if (g.residual) {
      float r[4];
      unpack(load_pack<DT, 4>((const E*)g.residual + m * g.ldr + c, n), r);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += r[i];
    }
    store_pack<DT, 4>((E*)g.y + m * g.ldy + c, pack<DT, 4>(v), n);
  }
}

__device__ __forceinline__ void add_bias4(const LinearArgs& g, int64_t c, int n, float (&v)[4]) {
  if (!g.bias) return;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) v[i] += load_any(g.bias, c + i, g.bias_dt);
}

// Which tile a workgroup takes.  Workgroups go to the 8 XCDs in turn, so
// workgroup i of an XCD is i * 8 + xcd; each XCD gets a run of consecutive
// tiles, and tiles run down 8 rows before the next column, so that what
// its L2 holds of A and B is used by its neighbours.
__device__ __forceinline__ void tile_of(int tiles_m, int tiles_n, int& tm, int& tn) {
  const int n = tiles_m * tiles_n, b = blockIdx.x;
  const int per = n / 8, rest = n % 8, xcd = b % 8;
  const int t = xcd * per + (xcd < rest ? xcd : rest) + b / 8;
  constexpr int kDown = 8;
  const int group = t / (kDown * tiles_n), first = group * kDown;
  const int down = tiles_m - first < kDown ? tiles_m - first : kDown;
  const int in = t - group * kDown * tiles_n;
  tm = first + in % down;
  tn = in / down;
}

template <int DT, int BM, int BN, int BK, int WM, int WN, int LA, int LB, int STAGES,
          bool DIRECT, int WAVES_EU>
__global__ __launch_bounds__(WM* WN * 64, WAVES_EU) void linear_kernel(LinearArgs g) {
  constexpr int NW = WM * WN;
  using TA = Tile<BM, BK, LA, NW>;
  using TB = Tile<BN, BK, LB, NW>;
  using F = typename Mfma<DT>::frag;
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  constexpr int kStage = TA::kBytes + TB::kBytes;
  __shared__ __attribute__((aligned(1024))) char smem[STAGES * kStage];
  lds_char* const lds = (lds_char*)smem;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  int tm, tn;
  tile_of(g.tiles_m, g.tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int have_m = g.M - m0 < BM ? (int)(g.M - m0) : BM;
  const int have_n = g.N - n0 < BN ? (int)(g.N - n0) : BN;

  // this split's steps of BK; the last of all may be a part of one
  const int64_t steps = (g.K + BK - 1) / BK;
  const int64_t per = (steps + g.splits - 1) / g.splits;
  const int64_t s0 = blockIdx.y * per;
  int64_t s1 = s0 + per < steps ? s0 + per : steps;
  const int64_t a_step = (LA == 0 ? BK : BK * g.lda) * 2;
  const int64_t b_step = (LB == 0 ? BK : BK * g.ldb) * 2;
  const char* a = (const char*)g.a + (LA == 0 ? m0 * g.lda : m0) * 2;
  const char* b = (const char*)g.b + (LB == 0 ? n0 * g.ldb : n0) * 2;

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  auto compute = [&](int stage) {
    const lds_char* const ta = lds + stage * kStage;
    const lds_char* const tb = ta + TA::kBytes;
#pragma unroll
    for (int kk = 0; kk < BK / 32; ++kk) {
      F fa[FM], fb[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j)
        fb[j] = TB::template frag<F>(tb, wn * (BN / WN) + j * 16, kk, lane);
#pragma unroll
      for (int i = 0; i < FM; ++i)
        fa[i] = TA::template frag<F>(ta, wm * (BM / WM) + i * 16, kk, lane);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = Mfma<DT>::run(fb[j], fa[i], acc[i][j]);
    }
  };

  const int tail = (int)(g.K % BK);
  if (s0 < s1) {
    u32x4 va[TA::kPerWave], vb[TB::kPerWave];
    if (s1 == steps && tail) {  // the part of a step, before the others
      s1 -= 1;
      TA::fetch(a + s1 * a_step, g.lda, have_m, tail, wave, lane, va);
      TB::fetch(b + s1 * b_step, g.ldb, have_n, tail, wave, lane, vb);
      TA::put(lds, wave, lane, va);
      TB::put(lds + TA::kBytes, wave, lane, vb);
      __syncthreads();
      compute(0);
      __syncthreads();
    }
    a += s0 * a_step;
    b += s0 * b_step;
    const int n = (int)(s1 - s0);
    if constexpr (DIRECT) {
      constexpr int kPer = TA::kPerWave + TB::kPerWave;
      uint32_t oa[TA::kPerWave], ob[TB::kPerWave];
      TA::offsets(g.lda, have_m, wave, lane, oa);
      TB::offsets(g.ldb, have_n, wave, lane, ob);
      int put = 0;  // the stage that the next load fills
      auto issue = [&] {
        const uint32_t at = lds0 + put * kStage;
        TA::load(a, oa, at, wave);
        TB::load(b, ob, at + TA::kBytes, wave);
        a += a_step;
        b += b_step;
        put = put + 1 == STAGES ? 0 : put + 1;
      };
      for (int t = 0; t < STAGES - 1 && t < n; ++t) issue();
      int get = 0;
      for (int t = 0; t < n; ++t) {
        // step t has landed (the loads of up to STAGES - 2 later steps may
        // be in flight), and the stage that is filled next is read out
        if (t + STAGES - 2 < n)
          wait_loads<(STAGES - 2) * kPer>();
        else
          wait_loads<0>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");  // no LDS read moves above the barrier
        if (t + STAGES - 1 < n) issue();
        compute(get);
        get = get + 1 == STAGES ? 0 : get + 1;
      }
    } else {
      if (n > 0) {
        TA::fetch(a, g.lda, have_m, BK, wave, lane, va);
        TB::fetch(b, g.ldb, have_n, BK, wave, lane, vb);
        TA::put(lds, wave, lane, va);
        TB::put(lds + TA::kBytes, wave, lane, vb);
      }
      __syncthreads();
      for (int t = 0; t < n; ++t) {
        a += a_step;
        b += b_step;
        if (t + 1 < n) {
          TA::fetch(a, g.lda, have_m, BK, wave, lane, va);
          TB::fetch(b, g.ldb, have_n, BK, wave, lane, vb);
        }
        compute(t & 1);
        if (t + 1 < n) {
          lds_char* const to = lds + ((t + 1) & 1) * kStage;
          TA::put(to, wave, lane, va);
          TB::put(to + TA::kBytes, wave, lane, vb);
        }
        __syncthreads();
      }
    }
  }

  // lane: row lane & 15 of each 16 x 16 tile, columns 4 (lane >> 4) .. + 3
  const int64_t row0 = m0 + wm * (BM / WM) + (lane & 15);
  const int64_t col0 = n0 + wn * (BN / WN) + (lane >> 4) * 4;
  if (g.partial) {
    float* const out = g.partial + (int64_t)blockIdx.y * g.M * g.N;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int64_t m = row0 + i * 16;
      if (m >= g.M) continue;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int64_t c = col0 + j * 16;
        const int n = g.N - c < 4 ? (int)(g.N - c) : 4;
        float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
        store_pack<kFP32, 4>(out + m * g.N + c, pack<kFP32, 4>(v), n);
      }
    }
    return;
  }
  const float limit = save_limit(DT);
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t m = row0 + i * 16;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int64_t c = col0 + j * 16;
      const int n = g.N - c < 4 ? (int)(g.N - c) : 4;
      float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
      add_bias4(g, c, n, v);
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i][j][q] = v[q];
    }
    if constexpr (FN % 2 == 0) {
      if (g.codes) {
#pragma unroll
        for (int j = 0; j < FN; j += 2) {
          // 32 columns: two tiles of the four lanes with this row
          float amax = 0.0f;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (col0 + (j + h) * 16 + q < g.N)
                amax = __builtin_fmaxf(amax, save_mag(acc[i][j + h][q], limit));
          amax = __builtin_fmaxf(amax, __shfl_xor(amax, 16));
          amax = __builtin_fmaxf(amax, __shfl_xor(amax, 32));
          const int s = save_scale(amax);
          const float down = scale_down(s);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int64_t c = col0 + (j + h) * 16;
            const int n = g.N - c < 4 ? (int)(g.N - c) : 4;
            Codes<4> q;
            q.w[0] = encode4(save_scaled(acc[i][j + h][0], limit, down),
                             save_scaled(acc[i][j + h][1], limit, down),
                             save_scaled(acc[i][j + h][2], limit, down),
                             save_scaled(acc[i][j + h][3], limit, down));
            if (m < g.M && n > 0) store_codes<4>(g.codes + m * g.N + c, q, n);
          }
          const int64_t c = col0 + j * 16;
          if (m < g.M && c < g.N && (lane >> 4) == 0)
            g.scales[m * ((g.N + kBlock - 1) / kBlock) + c / kBlock] = (uint8_t)s;
        }
      }
    }
    if (m >= g.M) continue;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int64_t c = col0 + j * 16;
      const int n = g.N - c < 4 ? (int)(g.N - c) : 4;
      float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
      if (n > 0) finish4<DT>(g, m, c, n, v);
    }
  }
}

// The runs' sums added in run order, then the epilogue: four columns a
// lane, eight neighbouring lanes for a checkpoint block.
template <int DT>
__global__ __launch_bounds__(256) void linear_finish_kernel(LinearArgs g) {
  const int64_t quads = (g.N + kBlock - 1) / kBlock * (kBlock / 4);  // of a row
  const int64_t total = quads * g.M;
  const float limit = save_limit(DT);
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total;
       t += (int64_t)gridDim.x * 256) {
    const int64_t m = t / quads, c = (t - m * quads) * 4;
    const int n = g.N - c < 4 ? (int)(g.N - c) : 4;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (n > 0) {
      const float* p = g.partial + m * g.N + c;
      unpack(load_pack<kFP32, 4>(p, n), v);
#pragma unroll 4
      for (int s = 1; s < g.splits; ++s) {
        float u[4];
        unpack(load_pack<kFP32, 4>(p + s * g.M * g.N, n), u);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += u[i];
      }
      add_bias4(g, c, n, v);
    }
    if (g.codes) {  // the eight lanes of a block are in the loop together
      Codes<4> q;
      const int s = encode<4>(v, n, limit, q);
      if (n > 0) store_codes<4>(g.codes + m * g.N + c, q, n);
      if (c % kBlock == 0) g.scales[m * (quads / 8) + c / kBlock] = (uint8_t)s;
    }
    if (n > 0) finish4<DT>(g, m, c, n, v);
  }
}

// ------------------------------------------------------------ variants
// Tile sizes, workgroup shapes and how they are picked: linear_plan.
enum { kTileBig = 0, kTileMid = 1, kTileSmall = 2, kTileFew = 3, kTiles = 4 };
struct TileShape {
  int bm, bn, bk, waves;
  bool pairs;  // a wave holds whole checkpoint blocks
};
constexpr TileShape kTileShape[kTiles] = {
    {256, 256, 64, 8, true}, {128, 128, 64, 4, true}, {64, 64, 64, 4, true}, {16, 64, 128, 4, false}};

template <int DT, int LA, int LB>
hipError_t linear_launch_tile(int tile, bool direct, const LinearArgs& g, hipStream_t s) {
  const dim3 grid((uint32_t)(g.tiles_m * g.tiles_n), (uint32_t)g.splits);
  if (direct) {
    switch (tile) {
      case kTileBig:
        linear_kernel<DT, 256, 256, 64, 2, 4, LA, LB, 2, true, 2><<<grid, 512, 0, s>>>(g);
        break;
      case kTileMid:
        linear_kernel<DT, 128, 128, 64, 2, 2, LA, LB, 2, true, 2><<<grid, 256, 0, s>>>(g);
        break;
      case kTileSmall:
        linear_kernel<DT, 64, 64, 64, 2, 2, LA, LB, 3, true, 2><<<grid, 256, 0, s>>>(g);
        break;
      default:
        linear_kernel<DT, 16, 64, 128, 1, 4, LA, LB, 3, true, 2><<<grid, 256, 0, s>>>(g);
    }
  } else {
    switch (tile) {
      case kTileMid:
        linear_kernel<DT, 128, 128, 64, 2, 2, LA, LB, 2, false, 2><<<grid, 256, 0, s>>>(g);
        break;
      case kTileSmall:
        linear_kernel<DT, 64, 64, 64, 2, 2, LA, LB, 2, false, 2><<<grid, 256, 0, s>>>(g);
        break;
      default:
        linear_kernel<DT, 16, 64, 128, 1, 4, LA, LB, 2, false, 2><<<grid, 256, 0, s>>>(g);
    }
  }
  return hipGetLastError();
}

// One element type's products and the kernel that finishes split ones.
template <int DT>
hipError_t linear_launch(int tile, bool direct, int la, int lb, const LinearArgs& g,
                         hipStream_t s) {
  hipError_t e;
  if (la == 0 && lb == 0)
    e = linear_launch_tile<DT, 0, 0>(tile, direct, g, s);
  else if (la == 0)
    e = linear_launch_tile<DT, 0, 1>(tile, direct, g, s);
  else
    e = linear_launch_tile<DT, 1, 1>(tile, direct, g, s);
  if (e != hipSuccess || !g.partial) return e;
  const int64_t lanes = (g.N + kBlock - 1) / kBlock * (kBlock / 4) * g.M;
  const int64_t blocks = (lanes + 255) / 256;
  linear_finish_kernel<DT><<<(uint32_t)(blocks < 65536 ? blocks : 65536), 256, 0, s>>>(g);
  return hipGetLastError();
}

hipError_t linear_launch_fp16(int tile, bool direct, int la, int lb, const LinearArgs& g,
                              hipStream_t s);
hipError_t linear_launch_bf16(int tile, bool direct, int la, int lb, const LinearArgs& g,
                              hipStream_t s);

}  // namespace mmaops
#endif
