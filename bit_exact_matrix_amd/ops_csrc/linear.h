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
// transposing LDS read, so that no operand is rearranged in memory (only
// one whose rows do not start on 16 bytes is copied to rows that do).
//
// Kernels.  linear_wide_kernel (256 x 256 and 128 x 128 tiles, a loop laid
// out by hand) for most products; linear_kernel for small tiles of 64 x 64
// and for few rows (16 x 64, also through registers where an operand allows
// no direct load); linear_rows_kernel for up to 16 rows in one launch.
// Where there are few tiles, K is split over workgroups and
// linear_finish_kernel adds the runs in order.
//
// LDS banks.  A layout-0 tile row is BK elements; 16-byte chunk c of row r
// is kept at chunk c ^ (r & 7), so that the rows of a fragment read spread
// over the banks.  A layout-1 tile row is one k with R columns; 32-byte
// slot s of row k is kept at s ^ g(k), with g taking 8 values over the 8
// rows that half a wave reads at once.  (Measured: no bank conflicts.)  The permutation is applied
// to the global address of each lane, as the LDS side of a direct load is
// always lane after lane.
//
// The matrix instruction takes B's fragment first: each lane then holds
// four neighbouring columns of one row of C.
#ifndef MMAOPS_LINEAR_H
#define MMAOPS_LINEAR_H

#include <type_traits>

#include "ops_common.h"
#include "plan.h"

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
  int grid_x;  // few rows: tiles of one z of the grid
  // the last whole step goes through registers too: its last row's last
  // chunk would pass the end of an operand
  int guard;
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
// The instruction set asks for one wait state between a write of M0 and the
// load that uses it, which nothing inserts inside an asm block: the s_nop.
__device__ __forceinline__ void load_to_lds(const char* base, uint32_t off, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %2\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %0, %1"
      :
      : "v"(off), "s"(base), "s"(lds)
      : "memory", "m0");
}

// A wave-uniform address, in scalar registers whatever the compiler keeps
// it in.
__device__ __forceinline__ const char* uniform(const char* p) {
  const uint64_t v = (uint64_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (const char*)((uint64_t)hi << 32 | lo);
}

// fn(integral_constant 0), .. fn(integral_constant N - 1)
template <int N, typename FN>
__device__ __forceinline__ void static_for(FN fn) {
  if constexpr (N > 0) {
    static_for<N - 1>(fn);
    fn(std::integral_constant<int, N - 1>{});
  }
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
    if constexpr (LAYOUT == 0) return r & 7;
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
  // past the matrix (`have` rows are there) repeat the last one, and a
  // chunk may pass the row's end: what they give is never stored
  static __device__ __forceinline__ void offsets(int64_t ld, int have, int wave, int lane,
                                                 uint32_t (&off)[kPerWave]) {
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) {
      int row, chunk;
      place((wave * kPerWave + i) * 64 + lane, row, chunk);
      if constexpr (LAYOUT == 0)
        row = row < have ? row : have - 1;
      else
        chunk = chunk * 8 < have ? chunk : (have - 1) / 8;
      off[i] = (uint32_t)(row * ld * 2) + chunk * 16;
    }
  }
  static __device__ __forceinline__ void load(const char* base, const uint32_t (&off)[kPerWave],
                                              uint32_t lds, int wave) {
#pragma unroll
    for (int i = 0; i < kPerWave; ++i)
      load_to_lds(uniform(base), off[i], lds + (wave * kPerWave + i) * 1024);
  }

  // The same through registers, for any alignment and for a tile with only
  // `kn` of its BK (the rest 0): `have` rows, in parts where a chunk passes
  // an edge.
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
        } else if (n > 0) {
          uint32_t w[4];
          load_part<4, 2>(p, n * 2, w);
          v[i] = u32x4{w[0], w[1], w[2], w[3]};
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

  // Fragment i, rows r0 + 16 i .. + 15, for k in [32 kk, 32 kk + 32): the
  // lane has row r0 + 16 i + (lane & 15) and 8 k from 8 (lane >> 4).  The
  // swaps depend on the lane alone, so an address is one per-lane base, an
  // exclusive or and constants (r0 is a multiple of the rows that the
  // wave's fragments span, a power of two, so r0 / 16 and i share no bit).
  static __device__ __forceinline__ uint32_t base(int r0, int lane) {
    if constexpr (LAYOUT == 0) {
      const int row = r0 + (lane & 15);
      return row * (BK * 2) + (((lane >> 4) ^ swap_of(row)) * 16);
    } else {
      const int k = (lane >> 4) * 8 + ((lane & 15) >> 2);
      return k * (R * 2) + (((r0 / 16) ^ swap_of(k)) * 32) + (lane & 3) * 8;
    }
  }
  template <typename F>
  static __device__ __forceinline__ F frag(const lds_char* tile, uint32_t base, int kk, int i) {
    if constexpr (LAYOUT == 0) {
      // kk & 1 is a chunk bit that the swap reaches, kk >> 1 one above
      return *(const __attribute__((address_space(3))) F*)(tile + (base ^ ((kk & 1) * 64)) +
                                                           (kk >> 1) * 128 + i * 16 * BK * 2);
    } else {
      using s4 = __attribute__((ext_vector_type(4))) short;
      union {
        s4 h[2];
        F f;
      } u;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        u.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s4*)(tile + (base ^ (i * 32)) +
                                                    (kk * 32 + h * 4) * (R * 2)));
      return u.f;
    }
  }
};

// ------------------------------------------------------------ epilogue
// Pre-activation, activation, residual and store of V columns (n of them
// there, V where FULL) of U rows m, m + step, ..; `res` has the residual's
// elements where it is of the operands' type.
template <int DT, int V, int U, bool FULL>
__device__ __forceinline__ void finish(const LinearArgs& g, int64_t m, int step, int64_t c, int n,
                                       float (&v)[U * V], const Pack<DT, V> (&res)[U]) {
  using E = elem_t<DT>;
  auto row = [&](int u, float (&o)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = v[u * V + i];
  };
  auto there = [&](int u) { return FULL || (m + u * step < g.M && n > 0); };
  const int k = FULL ? V : n;
  if (g.z) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float o[V];
      row(u, o);
      if (there(u))
        store_pack<DT, V>((E*)g.z + (m + u * step) * g.ldz + c, pack<DT, V>(o), k);
    }
  }
  act_all(v, g.act, act_apply);
  if (g.out_dt != kFP32) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float o[V], r[V];
      row(u, o);
      if (g.residual) {
        unpack(res[u], r);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] += r[i];
      }
      if (there(u))
        store_pack<DT, V>((E*)g.y + (m + u * step) * g.ldy + c, pack<DT, V>(o), k);
    }
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!there(u)) continue;
      float o[V], r[V];
      row(u, o);
      if (g.residual) {
        unpack(load_pack<kFP32, V>((const float*)g.residual + (m + u * step) * g.ldr + c, k), r);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] += r[i];
      }
      store_pack<kFP32, V>((float*)g.y + (m + u * step) * g.ldy + c, pack<kFP32, V>(o), k);
    }
  }
}

template <int V>
__device__ __forceinline__ void load_bias(const LinearArgs& g, int64_t c, int n, float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i)
    v[i] = g.bias && i < n ? load_any(g.bias, c + i, g.bias_dt) : 0.0f;
}

// A wave's FM x FN fragments of sums, whose first element is C's (m0, n0),
// to their place: the partial sums of a split product, or the output.  They
// go through LDS (the wave's own part of it, no barrier), PASS fragment
// rows at a time, so that a lane then has 8 neighbouring columns and
// neighbouring lanes a row: whole 16-byte stores, and 4 lanes for a
// checkpoint block.  A row's 16 bytes of padding spread the 16 rows of a
// fragment over the banks.  A lane takes four rows at once, so that their
// LDS reads and functions overlap, and has the next four rows' residual on
// its way meanwhile: with one wave a SIMD nothing else hides these.
template <int FN, int PASS>
constexpr int kStoreBytes = PASS * 16 * (FN * 64 + 16);

template <int DT, int FM, int FN, int PASS>
__device__ __forceinline__ void store_tile(const LinearArgs& g, const f32x4 (&acc)[FM][FN],
                                           lds_char* mem, int64_t m0, int64_t n0, int lane,
                                           int split) {
  using E = elem_t<DT>;
  using lds_f4 = __attribute__((address_space(3))) f32x4;
  constexpr int kRow = FN * 64 + 16;
  constexpr int kLanes = FN * 2, kRows = 64 / kLanes;  // lanes a row, rows at once
  constexpr int kPassRows = PASS * 16;
  constexpr int kTurns = (kPassRows + kRows - 1) / kRows;
  constexpr int U = kTurns < 4 ? kTurns : 4;
  const int64_t c = n0 + (lane % kLanes) * 8;
  const int n = g.N - c < 8 ? (int)(g.N - c) : 8;
  const bool full = m0 + FM * 16 <= g.M && n0 + FN * 16 <= g.N;
  auto put = [&](int i) {
#pragma unroll
    for (int h = 0; h < PASS; ++h)
#pragma unroll
      for (int j = 0; j < FN; ++j)
        *(lds_f4*)(mem + (h * 16 + (lane & 15)) * kRow + j * 64 + (lane >> 4) * 16) =
            acc[i + h][j];
  };
  auto get = [&](int r, float* v) {
    const lds_f4* const p = (const lds_f4*)(mem + r * kRow + (lane % kLanes) * 32);
    const f32x4 lo = p[0], hi = p[1];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] = lo[q];
      v[4 + q] = hi[q];
    }
  };
  if (g.partial) {
    float* const out = g.partial + (int64_t)split * g.M * g.N + c;
#pragma unroll
    for (int i = 0; i < FM; i += PASS) {
      put(i);
#pragma unroll 2
      for (int r = lane / kLanes; r < kPassRows; r += kRows) {
        const int64_t m = m0 + i * 16 + r;
        float v[8];
        get(r, v);
        if (m < g.M && n > 0) store_pack<kFP32, 8>(out + m * g.N, pack<kFP32, 8>(v), n);
      }
    }
    return;
  }
  float bias[8];
  load_bias<8>(g, c, n, bias);
  const bool fetches = g.residual && g.out_dt != kFP32;
  int64_t mr = m0 + lane / kLanes;  // the row whose residual is loaded next
  const int64_t m1 = m0 + FM * 16 < g.M ? m0 + FM * 16 : g.M;
  Pack<DT, 8> ahead[U];
  auto fetch = [&] {
    if (!fetches) return;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (mr < m1) ahead[u] = load_pack<DT, 8>((const E*)g.residual + mr * g.ldr + c, n);
      mr += kRows;
    }
  };
  fetch();
#pragma unroll
  for (int i = 0; i < FM; i += PASS) {
    put(i);
#pragma unroll 1
    for (int r = lane / kLanes; r < kPassRows; r += U * kRows) {
      const int64_t m = m0 + i * 16 + r;
      float v[U * 8];
#pragma unroll
      for (int u = 0; u < U; ++u) get(r + u * kRows, v + u * 8);
      Pack<DT, 8> res[U];
#pragma unroll
      for (int u = 0; u < U; ++u) res[u] = ahead[u];
      fetch();
#pragma unroll
      for (int q = 0; q < U * 8; ++q) v[q] += bias[q % 8];
      if constexpr (FN % 2 == 0) {
        if (g.codes) {  // a row's lanes are here together
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int64_t mu = m + u * kRows;
            float o[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] = v[u * 8 + q];
            Codes<8> q;
            const int s = encode<DT, 8>(o, n, q);
            if (mu < g.M && n > 0) {
              store_codes<8>(g.codes + mu * g.N + c, q, n);
              if (c % kBlock == 0)
                g.scales[mu * ((g.N + kBlock - 1) / kBlock) + c / kBlock] = (uint8_t)s;
            }
          }
        }
      }
      if (full)
        finish<DT, 8, U, true>(g, m, kRows, c, 8, v, res);
      else
        finish<DT, 8, U, false>(g, m, kRows, c, n, v, res);
    }
  }
}

// Which tile workgroup b takes.  Workgroups go to the 8 XCDs in turn, so
// workgroup i of an XCD is i * 8 + xcd; each XCD gets a run of consecutive
// tiles, and tiles run down 8 rows before the next column, so that what
// its L2 holds of A and B is used by its neighbours.
__device__ __forceinline__ void tile_of(int tiles_m, int tiles_n, int b, int& tm, int& tn) {
  const int n = tiles_m * tiles_n;
  const int per = n / 8, rest = n % 8, xcd = b % 8;
  const int t = xcd * per + (xcd < rest ? xcd : rest) + b / 8;
  constexpr int kDown = 8;
  const int group = t / (kDown * tiles_n), first = group * kDown;
  const int down = tiles_m - first < kDown ? tiles_m - first : kDown;
  const int in = t - group * kDown * tiles_n;
  tm = first + in % down;
  tn = in / down;
}

template <int BM, int BN, int BK, int STAGES>
constexpr int kRingBytes = STAGES * (BM + BN) * BK * 2;

// The small tiles, their loop left to the compiler: several workgroups on a
// CU hide each other's waits.  A ring of STAGES steps, one barrier a step;
// DIRECT: direct loads, else through registers.
template <int DT, int BM, int BN, int BK, int WM, int WN, int LA, int LB, int STAGES,
          bool DIRECT>
__device__ __forceinline__ void small_product(const LinearArgs& g, int block, int split,
                                              char* smem) {
  constexpr int NW = WM * WN;
  using TA = Tile<BM, BK, LA, NW>;
  using TB = Tile<BN, BK, LB, NW>;
  using F = typename Mfma<DT>::frag;
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  constexpr int kStage = TA::kBytes + TB::kBytes;
  lds_char* const lds = (lds_char*)smem;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  int tm, tn;
  tile_of(g.tiles_m, g.tiles_n, block, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int have_m = g.M - m0 < BM ? (int)(g.M - m0) : BM;
  const int have_n = g.N - n0 < BN ? (int)(g.N - n0) : BN;

  // this split's steps of BK; the last of all may be a part of one
  const int64_t steps = (g.K + BK - 1) / BK;
  const int64_t per = (steps + g.splits - 1) / g.splits;
  const int64_t s0 = split * per;
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
  const uint32_t base_a = TA::base(wm * (BM / WM), lane), base_b = TB::base(wn * (BN / WN), lane);

  auto compute = [&](int stage) {
    const lds_char* const ta = lds + stage * kStage;
    const lds_char* const tb = ta + TA::kBytes;
#pragma unroll
    for (int kk = 0; kk < BK / 32; ++kk) {
      F fa[FM], fb[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) fb[j] = TB::template frag<F>(tb, base_b, kk, j);
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[i] = TA::template frag<F>(ta, base_a, kk, i);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = Mfma<DT>::run(fb[j], fa[i], acc[i][j]);
    }
  };

  const int tail = g.K % BK ? (int)(g.K % BK) : g.guard ? BK : 0;
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

  constexpr int kPass = FM > 1 ? 2 : 1;
  static_assert(NW * kStoreBytes<FN, kPass> <= STAGES * kStage, "the epilogue's LDS");
  __syncthreads();
  store_tile<DT, FM, FN, kPass>(g, acc, lds + wave * kStoreBytes<FN, kPass>, m0 + wm * (BM / WM),
                                n0 + wn * (BN / WN), lane, split);
}

template <int DT, int BM, int BN, int BK, int WM, int WN, int LA, int LB, int STAGES,
          bool DIRECT, int WAVES_EU>
__global__ __launch_bounds__(WM* WN * 64, WAVES_EU) void linear_kernel(LinearArgs g) {
  __shared__ __attribute__((aligned(1024))) char smem[kRingBytes<BM, BN, BK, STAGES>];
  const int block = (int)(blockIdx.x + blockIdx.z * (uint32_t)g.grid_x);
  if (block >= g.tiles_m * g.tiles_n) return;  // the whole workgroup
  small_product<DT, BM, BN, BK, WM, WN, LA, LB, STAGES, DIRECT>(g, block, blockIdx.y, smem);
}

// A small backward pass's second launch: the tiles of dz W^T (layouts 0, LB),
// then those of X^T dz (1, 1), then the bias gradient's column sums, 64
// columns a workgroup; all need only the first launch's dz and partial sums.
// Launches bound such a pass, so three are one (fp16, gelu, the whole pass on
// the GPU, apart and together: 299 x 260 x 640 21.5 us and 13.8, 512 x 512 x
// 512 17.7 and 10.3, 1024 x 1024 x 1024 25.5 and 16.7).
struct PairArgs {
  LinearArgs dx, dw;
  const float* partial;  // [count][cols]
  void* dbias;           // NULL: none
  int64_t cols;
  int count, dbias_dt;
};

template <int DT, int LB>
__global__ __launch_bounds__(256, 2) void linear_pair_kernel(PairArgs p) {
  __shared__ __attribute__((aligned(1024))) char smem[kRingBytes<64, 64, 64, 3>];
  const int n1 = p.dx.tiles_m * p.dx.tiles_n, n2 = p.dw.tiles_m * p.dw.tiles_n;
  const int b = blockIdx.x;
  if (b < n1) {
    small_product<DT, 64, 64, 64, 2, 2, 0, LB, 3, true>(p.dx, b, 0, smem);
  } else if (b < n1 + n2) {
    small_product<DT, 64, 64, 64, 2, 2, 1, 1, 3, true>(p.dw, b - n1, 0, smem);
  } else {
    // in the runs and the order of column_sum_kernel, for the same bits
    float(&meet)[16][64] = *(float(*)[16][64])smem;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)(b - n1 - n2) * 64 + lane;
    const int run = (p.count + 15) / 16;
    // four of the sixteen runs a wave, side by side; past a run's end + 0
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < p.cols) {
#pragma unroll 4
      for (int q = 0; q < run; ++q) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = (wave * 4 + i) * run + q;
          s[i] += row < p.count ? p.partial[row * p.cols + c] : 0.0f;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) meet[wave * 4 + i][lane] = s[i];
    __syncthreads();
    if (wave == 0 && c < p.cols) {
      float sum = meet[0][lane];
#pragma unroll
      for (int r = 1; r < 16; ++r) sum += meet[r][lane];
      store_any(p.dbias, c, sum, p.dbias_dt);
    }
  }
}

// The large tiles: four waves, one for each SIMD, with a quarter of the tile
// each.  A wave of 128 x 128 (256 x 256 tile) reads 1 KiB of LDS for 16
// matrix instructions, where 128 x 64 reads 1.5 KiB: with eight waves LDS
// reads and the tile's arrival would take as many cycles as the products.
// With one wave a SIMD nothing else hides a wait, so the loop is laid out
// by hand (times below: 256 x 256, two stages): each LDS read and each load
// sits alone behind a matrix instruction, as a lone wave issues one
// instruction every 4 cycles and a product takes 16.  A step of BK = 64
// runs in two halves of 64 products from registers:
//   first half    the fragments of this step's second half are read; when
//                 they are there (slot 34) a barrier frees the stage, and
//                 the loads of the step after next begin to fill it
//   (barrier: the next step has landed)
//   second half   the fragments of the next step's first half are read, and
//                 the loads go on
// so a load has 1,200 to 2,400 cycles to land.  Loads every 4 slots or fewer
// wait for the vector memory pipe (8192^3: every 2, 844 us, 4, 792, 5, 782).
// What is left: 8192^3 bf16 takes 768 us (X W), 751 (X W^T) and 774 (X^T
// dY), 1.42 to 1.46 PFLOP/s, at 1.6 to 1.8 GHz under this load with the matrix
// cores busy 71% (X W) and 76% (X W^T) of the cycles.  A row of 64 elements is
// a whole 128-byte line; steps of 32 with a ring of four stages kept the
// vector memory pipe busier than the products (8192^3, both operands with K
// fastest: 922 us against 856).
template <int DT, int LA, int LB, int BM, int BN, int STAGES>
__global__ __launch_bounds__(256, 1) void linear_wide_kernel(LinearArgs g) {
  constexpr int BK = 64, NW = 4, FM = BM / 32, FN = BN / 32;
  using TA = Tile<BM, BK, LA, NW>;
  using TB = Tile<BN, BK, LB, NW>;
  using F = typename Mfma<DT>::frag;
  constexpr int kStage = TA::kBytes + TB::kBytes;
  constexpr int kLoads = TA::kPerWave + TB::kPerWave;  // of a wave and step
  constexpr int kPass = FM < 8 ? 2 : 4;  // of the epilogue
  constexpr int kBytes = STAGES * kStage > NW * kStoreBytes<FN, kPass>
                             ? STAGES * kStage
                             : NW * kStoreBytes<FN, kPass>;
  __shared__ __attribute__((aligned(1024))) char smem[kBytes];
  lds_char* const lds = (lds_char*)smem;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  int tm, tn;
  tile_of(g.tiles_m, g.tiles_n, blockIdx.x, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int have_m = g.M - m0 < BM ? (int)(g.M - m0) : BM;
  const int have_n = g.N - n0 < BN ? (int)(g.N - n0) : BN;
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
  const uint32_t base_a = TA::base(wm * (BM / 2), lane);
  const uint32_t base_b = TB::base(wn * (BN / 2), lane) + TA::kBytes;

  const int tail = g.K % BK ? (int)(g.K % BK) : g.guard ? BK : 0;
  if (s0 < s1 && s1 == steps && tail) {  // the part of a step, before the others
    s1 -= 1;
    u32x4 va[TA::kPerWave], vb[TB::kPerWave];
    TA::fetch(a + s1 * a_step, g.lda, have_m, tail, wave, lane, va);
    TA::put(lds, wave, lane, va);
    TB::fetch(b + s1 * b_step, g.ldb, have_n, tail, wave, lane, vb);
    TB::put(lds + TA::kBytes, wave, lane, vb);
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const F fb = TB::template frag<F>(lds, base_b, kk, j);
#pragma unroll
        for (int i = 0; i < FM; ++i)
          acc[i][j] = Mfma<DT>::run(fb, TA::template frag<F>(lds, base_a, kk, i), acc[i][j]);
      }
    __syncthreads();
  }
  const int n = (int)(s1 - s0);
  if (n > 0) {
    a += s0 * a_step;
    b += s0 * b_step;
    uint32_t oa[TA::kPerWave], ob[TB::kPerWave];
    TA::offsets(g.lda, have_m, wave, lane, oa);
    TB::offsets(g.ldb, have_n, wave, lane, ob);
    // load i of a step, into the stage at `to`
    auto issue = [&](int i, uint32_t to) {
      if (i < TB::kPerWave)
        load_to_lds(uniform(b), ob[i], to + TA::kBytes + (wave * TB::kPerWave + i) * 1024);
      else
        load_to_lds(uniform(a), oa[i - TB::kPerWave],
                    to + (wave * TA::kPerWave + i - TB::kPerWave) * 1024);
    };
    // one step further; past the last one the same again (loaded, not used)
    int left = n;
    auto next = [&] {
      const bool more = --left > 0;
      a += more ? a_step : 0;
      b += more ? b_step : 0;
    };
    auto read = [&](F (&fa)[FM], F (&fb)[FN], int q, int kk, const lds_char* from) {
      if (q < FN)
        fb[q] = TB::template frag<F>(from, base_b, kk, q);
      else
        fa[q - FN] = TA::template frag<F>(from, base_a, kk, q - FN);
    };
    auto barrier = [] {
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    };
    // Products of a half, slots between reads and between loads, the slot
    // of the first barrier, and the loads before the second.
    constexpr int S = FM * FN, kRead = S >= 64 ? 2 : 1, kEvery = S >= 64 ? 5 : 2;
    constexpr int kFree = S >= 64 ? 34 : S >= 32 ? 20 : 12;
    constexpr int kFirst = (S - 1 - kFree - 2) / kEvery + 1;
    static_assert((FM + FN) * kRead <= kFree && (kLoads - kFirst) * kEvery < S, "slots");
    F a0[FM], b0[FN], a1[FM], b1[FN];
    uint32_t at = 0;  // this step's stage
    auto after = [](uint32_t stage) {
      return stage + kStage == STAGES * kStage ? 0u : stage + kStage;
    };
    auto first_half = [&] {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        acc[s / FN][s % FN] = Mfma<DT>::run(b0[s % FN], a0[s / FN], acc[s / FN][s % FN]);
        if (s % kRead == 0 && s / kRead < FM + FN) read(a1, b1, s / kRead, 1, lds + at);
        if (s == kFree) {
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          barrier();
        }
        if (s >= kFree + 2 && (s - kFree - 2) % kEvery == 0)
          issue((s - kFree - 2) / kEvery, lds0 + at);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    auto second_half = [&] {
      const lds_char* const from = lds + after(at);
#pragma unroll
      for (int s = 0; s < S; ++s) {
        acc[s / FN][s % FN] = Mfma<DT>::run(b1[s % FN], a1[s / FN], acc[s / FN][s % FN]);
        if (s % kRead == 0 && s / kRead < FM + FN) read(a0, b0, s / kRead, 0, from);
        if (s % kEvery == 1 && s / kEvery < kLoads - kFirst)
          issue(kFirst + s / kEvery, lds0 + at);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) issue(i, lds0 + s * kStage);
      next();
    }
    wait_loads<(STAGES - 1) * kLoads>();
    barrier();
#pragma unroll
    for (int q = 0; q < FM + FN; ++q) read(a0, b0, q, 0, lds);
    for (int t = 0; t < n; ++t) {
      first_half();
      wait_loads<(STAGES - 2) * kLoads + kFirst>();
      barrier();
      second_half();
      next();
      at = after(at);
    }
    wait_loads<0>();
  }
  __syncthreads();
  store_tile<DT, FM, FN, kPass>(g, acc, lds + wave * kStoreBytes<FN, kPass>,
                                m0 + wm * (BM / 2), n0 + wn * (BN / 2), lane, blockIdx.y);
}

// The end of a product of up to ROWS rows: BN columns' [wave][row][column]
// sums added in wave order, then the epilogue, four columns a lane.
template <int DT, int ROWS, int BN, int NW>
__device__ __forceinline__ void finish_rows(const LinearArgs& g, const lds_char* meet,
                                            int64_t n0) {
  using lds_f4 = __attribute__((address_space(3))) f32x4;
  constexpr int kMeet = ROWS * BN * 4;
  if (threadIdx.x >= ROWS * BN / 4) return;
  const int64_t m = threadIdx.x / (BN / 4), c = n0 + threadIdx.x % (BN / 4) * 4;
  const int have = g.N - c < 4 ? (int)(g.N - c) : 4;
  float v[4], bias[4];
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const f32x4 u = *(const lds_f4*)(meet + w * kMeet + threadIdx.x * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = w ? v[i] + u[i] : u[i];
  }
  load_bias<4>(g, c, have, bias);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] += bias[i];
  if constexpr (BN >= 32) {
    if (g.codes) {
      Codes<4> q;
      float o[4] = {v[0], v[1], v[2], v[3]};
      const int s = encode<DT, 4>(o, have, q);
      if (m < g.M && have > 0) {
        store_codes<4>(g.codes + m * g.N + c, q, have);
        if (c % kBlock == 0)
          g.scales[m * ((g.N + kBlock - 1) / kBlock) + c / kBlock] = (uint8_t)s;
      }
    }
  }
  Pack<DT, 4> res[1] = {};
  if (m < g.M && have > 0 && g.residual && g.out_dt != kFP32)
    res[0] = load_pack<DT, 4>((const elem_t<DT>*)g.residual + m * g.ldr + c, have);
  finish<DT, 4, 1, false>(g, m, 0, c, have, v, res);
}

// Up to 16 rows (a decoding step): what bounds it is reading the weight
// once, from as many CUs and with as much under way as there can be.  A
// workgroup takes BN = 16 columns (32 where z is saved, as a checkpoint
// block is) and all of K, shared out over its eight waves.  A wave issues
// the loads of its whole part of the weight at once, up to 16 KB, to LDS of
// its own (no barrier); its part of X goes to registers.  The waves' sums
// meet once, in wave order.  1 x 4096 x 4096 bf16, time on the GPU: W stored
// N x K 8.6 us (3.9 TB/s), K x N 13.2 us, where a row of the tile is only 32
// bytes (32 columns 13.6, 64 columns 14.9: fewer workgroups); K split over
// workgroups and joined by a second kernel takes 8.7 + 3.8 us and a second
// launch.
template <int DT, int LB, int BN>
__global__ __launch_bounds__(512, 2) void linear_rows_kernel(LinearArgs g) {
  constexpr int BK = 64, NW = 8, FN = BN / 16, kSteps = 8 / FN;  // steps at once
  using TB = Tile<BN, BK, LB, 1>;
  using F = typename Mfma<DT>::frag;
  using lds_f4 = __attribute__((address_space(3))) f32x4;
  constexpr int kPer = TB::kPerWave;
  __shared__ __attribute__((aligned(1024))) char smem[NW * kSteps * TB::kBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  lds_char* const lds = (lds_char*)smem + wave * kSteps * TB::kBytes;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
  int tm, tn;
  tile_of(1, (int)gridDim.x, blockIdx.x, tm, tn);
  const int64_t n0 = (int64_t)tn * BN;
  const int have_n = g.N - n0 < BN ? (int)(g.N - n0) : BN;
  const int64_t steps = g.K / BK, s0 = steps * wave / NW, s1 = steps * (wave + 1) / NW;
  const int64_t b_step = (LB == 0 ? BK : BK * g.ldb) * 2;
  const char* b = (const char*)g.b + (LB == 0 ? n0 * g.ldb : n0) * 2 + s0 * b_step;
  // rows past M repeat the last one: what they give is not stored
  const int64_t row = (lane & 15) < g.M ? (lane & 15) : g.M - 1;
  const char* x = (const char*)g.a + (row * g.lda + s0 * BK + (lane >> 4) * 8) * 2;
  uint32_t ob[kPer];
  TB::offsets(g.ldb, have_n, 0, lane, ob);
  const uint32_t base_b = TB::base(0, lane);
  f32x4 acc[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t s = s0; s < s1; s += kSteps) {
    const int n = s1 - s < kSteps ? (int)(s1 - s) : kSteps;
    F fx[kSteps][2];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // LDS is read out
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
      if (t >= n) continue;
      __builtin_memcpy(&fx[t][0], x + t * BK * 2, 16);
      __builtin_memcpy(&fx[t][1], x + t * BK * 2 + 64, 16);
    }
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
      if (t >= n) continue;
      TB::load(b, ob, lds0 + t * TB::kBytes, 0);
      b += b_step;
    }
    x += kSteps * BK * 2;
    static_for<kSteps>([&](auto step) {
      constexpr int t = decltype(step)::value;
      if (t >= n) return;
      if (n == kSteps)
        wait_loads<(kSteps - 1 - t) * kPer>();
      else
        wait_loads<0>();
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[j] = Mfma<DT>::run(
              TB::template frag<F>(lds + t * TB::kBytes, base_b, kk, j), fx[t][kk], acc[j]);
    });
  }
  // [wave][row][column] sums
  lds_char* const meet = (lds_char*)smem;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < FN; ++j)
    *(lds_f4*)(meet + wave * (16 * BN * 4) + (lane & 15) * BN * 4 + j * 64 + (lane >> 4) * 16) =
        acc[j];
  __syncthreads();
  finish_rows<DT, 16, BN, NW>(g, meet, n0);
}

// One or two rows against a weight stored K x N whose rows direct loads
// cannot take (odd lengths): in one launch, through registers.  A lane has 8
// columns of 8 consecutive rows of the weight, all on their way at once (up
// to 128 KB a workgroup), and its own sums of MR x 8 products.  The lanes' sums
// meet by swaps, the waves' in LDS in wave order.  A row's piece of 32 bytes costs
// a CU about 4 cycles and one of 128 bytes 5, so BN = 16 columns only while
// that gives each CU one workgroup, then 32, then 64 (1 x 4097 x 4096: 18.9,
// 15.2 and 23.2 us; 1 x 11009 x 4095: 39.9, 33.5 and 25.6).  One row, bf16,
// beside the weight copied to aligned rows or the tile of few rows through
// registers: N x K 1499 x 1023 8.7 us and 13.7, 2135 x 132 5.4 and 7.3, 4097
// x 4096 15.2 and 21.6.  Aligned weights: 4096 x 4096 14.8 here, 13.0 with K
// split over workgroups.  Four rows: more products and sums than registers,
// 11.7 and 14.0, 22.0 and 25.2, but 42 and 32 at 11009 x 4095.  The order of
// the sums goes with BN, so where z is saved as blocks of 32 columns a
// workgroup holds two times 16 (PARTS, of NW waves each), and the output's
// bits are those of a call that saves nothing.
template <int DT, int MR, int BN, int PARTS, int NW>
__global__ __launch_bounds__(PARTS* NW * 64) void linear_vec_kernel(LinearArgs g) {
  constexpr int kLanes = BN / 8, kAtOnce = NW * 64 / kLanes;  // runs of 8 rows
  constexpr int kCols = BN * PARTS;
  __shared__ __attribute__((aligned(16))) float smem[NW * MR * kCols];
  const int lane = threadIdx.x & 63;
  const int part = (threadIdx.x >> 6) / NW, wave = (threadIdx.x >> 6) % NW;
  int tm, tn;
  tile_of(1, (int)gridDim.x, blockIdx.x, tm, tn);
  const int64_t n0 = (int64_t)tn * kCols;
  const elem_t<DT>* const a = (const elem_t<DT>*)g.a;
  const int64_t c = n0 + part * BN + (lane % kLanes) * 8;
  const int n = g.N - c < 8 ? (int)(g.N - c) : 8;
  const elem_t<DT>* const b = (const elem_t<DT>*)g.b + c;
  float v[MR * 8];
#pragma unroll
  for (int i = 0; i < MR * 8; ++i) v[i] = 0.0f;
  for (int64_t k = (int64_t)((wave * 64 + lane) / kLanes) * 8; k < g.K; k += kAtOnce * 8) {
    const int have = g.K - k < 8 ? (int)(g.K - k) : 8;
    Pack<DT, 8> w[8], x[MR];
    if (n == 8 && have == 8) {
#pragma unroll
      for (int t = 0; t < 8; ++t) w[t] = load_pack<DT, 8>(b + (k + t) * g.ldb);
#pragma unroll
      for (int m = 0; m < MR; ++m) x[m] = load_pack<DT, 8>(a + m * g.lda + k);
    } else {
#pragma unroll
      for (int t = 0; t < 8; ++t) w[t] = load_pack<DT, 8>(b + (k + t) * g.ldb, t < have ? n : 0);
#pragma unroll
      for (int m = 0; m < MR; ++m) x[m] = load_pack<DT, 8>(a + m * g.lda + k, have);
    }
    float xv[MR][8];
#pragma unroll
    for (int m = 0; m < MR; ++m) unpack(x[m], xv[m]);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      float wv[8];
      unpack(w[t], wv);
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[m * 8 + i] = fmaf(wv[i], xv[m][t], v[m * 8 + i]);
    }
  }
  // over the wave's lanes of the same columns: the upper half keeps columns
  // 4 to 7, odd rows of 16 lanes 2 and 3 (6 and 7), then rows turned
#pragma unroll
  for (int m = 0; m < MR; ++m) {
    float h[4], q[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = swap_add32(v[m * 8 + i], v[m * 8 + 4 + i]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      q[i] = swap_add16(h[i], h[2 + i]);
      if constexpr (kLanes <= 2) q[i] += dpp<kRor2>(q[i]);
      if constexpr (kLanes <= 4) q[i] += dpp<kRor4>(q[i]);
      q[i] += dpp<kRor8>(q[i]);
    }
    if ((lane & 15) < kLanes) {
      float* const o = smem + (wave * MR + m) * kCols + part * BN + (lane & 15) * 8 +
                       (lane >> 5) * 4 + (lane >> 4 & 1) * 2;
      o[0] = q[0];
      o[1] = q[1];
    }
  }
  __syncthreads();
  finish_rows<DT, MR, kCols, NW>(g, (const lds_char*)smem, n0);
}

// The runs' sums added in run order, then the epilogue: four columns a
// lane, eight neighbouring lanes for a checkpoint block.
template <int DT>
__global__ __launch_bounds__(64) void linear_finish_kernel(LinearArgs g) {
  const int64_t quads = (g.N + kBlock - 1) / kBlock * (kBlock / 4);  // of a row
  const int64_t total = quads * g.M;
  for (int64_t t = (int64_t)blockIdx.x * 64 + threadIdx.x; t < total;
       t += (int64_t)gridDim.x * 64) {
    const int64_t m = t / quads, c = (t - m * quads) * 4;
    const int n = g.N - c < 4 ? (int)(g.N - c) : 4;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (n > 0) {
      // eight runs' sums on their way at once
      const float* p = g.partial + m * g.N + c;
      const int64_t run = g.M * g.N;
      for (int s0 = 0; s0 < g.splits; s0 += 8) {
        Pack<kFP32, 4> u[8];
#pragma unroll
        for (int s = 0; s < 8; ++s)
          u[s] = load_pack<kFP32, 4>(p + (s0 + s) * run, s0 + s < g.splits ? n : 0);
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          float w[4];
          unpack(u[s], w);
          if (s0 + s < g.splits) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = s0 + s ? v[i] + w[i] : w[i];
          }
        }
      }
      float bias[4];
      load_bias<4>(g, c, n, bias);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += bias[i];
    }
    if (g.codes) {  // the eight lanes of a block are in the loop together
      Codes<4> q;
      float o[4] = {v[0], v[1], v[2], v[3]};
      const int s = encode<DT, 4>(o, n, q);
      if (n > 0) store_codes<4>(g.codes + m * g.N + c, q, n);
      if (c % kBlock == 0) g.scales[m * (quads / 8) + c / kBlock] = (uint8_t)s;
    }
    Pack<DT, 4> res[1];
    if (n > 0 && g.residual && g.out_dt != kFP32)
      res[0] = load_pack<DT, 4>((const elem_t<DT>*)g.residual + m * g.ldr + c, n);
    finish<DT, 4, 1, false>(g, m, 0, c, n, v, res);
  }
}

// ------------------------------------------------------------ variants
template <int DT, int MR>
void vec_launch(const LinearArgs& g, hipStream_t s) {
  const auto grid = [&](int bn) { return (uint32_t)((g.N + bn - 1) / bn); };
  if (grid(16) > 256) {
    if (grid(32) <= 256)
      linear_vec_kernel<DT, MR, 32, 1, 16><<<grid(32), 1024, 0, s>>>(g);
    else
      linear_vec_kernel<DT, MR, 64, 1, 16><<<grid(64), 1024, 0, s>>>(g);
  } else if (g.codes) {
    linear_vec_kernel<DT, MR, 16, 2, 8><<<grid(32), 1024, 0, s>>>(g);
  } else {
    linear_vec_kernel<DT, MR, 16, 1, 8><<<grid(16), 512, 0, s>>>(g);
  }
}

template <int DT, int LA, int LB>
hipError_t linear_launch_tile(int tile, bool direct, const LinearArgs& g, hipStream_t s) {
  const dim3 grid((uint32_t)(g.tiles_m * g.tiles_n), (uint32_t)g.splits);
  switch (tile) {
    case kTileBig:
      linear_wide_kernel<DT, LA, LB, 256, 256, 2><<<grid, 256, 0, s>>>(g);
      break;
    case kTileMid:
      // One workgroup a CU: three stages, for the loads have only 32 products
      // a step to land behind.  More: two stages, so that two workgroups
      // share a CU and hide each other's waits (bf16, K = 4096: 256 tiles
      // 34.6 us with three, 43 with two; 512 tiles 64 and 59).
      if ((int64_t)grid.x * grid.y <= 256)
        linear_wide_kernel<DT, LA, LB, 128, 128, 3><<<grid, 256, 0, s>>>(g);
      else
        linear_wide_kernel<DT, LA, LB, 128, 128, 2><<<grid, 256, 0, s>>>(g);
      break;
    case kTileSmall:
      linear_kernel<DT, 64, 64, 64, 2, 2, LA, LB, 3, true, 2><<<grid, 256, 0, s>>>(g);
      break;
    case kTileRows:
      if constexpr (LA == 0) {
        if (g.codes)
          linear_rows_kernel<DT, LB, 32><<<dim3((uint32_t)((g.N + 31) / 32)), 512, 0, s>>>(g);
        else
          linear_rows_kernel<DT, LB, 16><<<dim3((uint32_t)((g.N + 15) / 16)), 512, 0, s>>>(g);
      }
      break;
    case kTileVec:
      if constexpr (LA == 0 && LB == 1) {
        if (g.M == 1)
          vec_launch<DT, 1>(g, s);
        else
          vec_launch<DT, 2>(g, s);
      }
      break;
    default: {
      // a grid has fewer than 2^32 lanes in x
      constexpr uint32_t kMost = 1u << 23;
      LinearArgs f = g;
      f.grid_x = (int)(grid.x < kMost ? grid.x : kMost);
      const dim3 few((uint32_t)f.grid_x, grid.y, (grid.x + kMost - 1) / kMost);
      if (direct)
        linear_kernel<DT, 16, 64, 128, 1, 4, LA, LB, 3, true, 2><<<few, 256, 0, s>>>(f);
      else
        linear_kernel<DT, 16, 64, 128, 1, 4, LA, LB, 2, false, 2><<<few, 256, 0, s>>>(f);
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
  const int64_t blocks = (lanes + 63) / 64;  // small ones: few outputs on many CUs
  linear_finish_kernel<DT><<<(uint32_t)(blocks < 65536 ? blocks : 65536), 64, 0, s>>>(g);
  return hipGetLastError();
}

template <int DT>
hipError_t pair_launch(int lb, const PairArgs& p, hipStream_t s) {
  const int64_t sums = p.dbias ? (p.cols + 63) / 64 : 0;
  const uint32_t grid = (uint32_t)((int64_t)p.dx.tiles_m * p.dx.tiles_n +
                                   (int64_t)p.dw.tiles_m * p.dw.tiles_n + sums);
  if (lb)
    linear_pair_kernel<DT, 1><<<grid, 256, 0, s>>>(p);
  else
    linear_pair_kernel<DT, 0><<<grid, 256, 0, s>>>(p);
  return hipGetLastError();
}

hipError_t pair_launch_fp16(int lb, const PairArgs& p, hipStream_t s);
hipError_t pair_launch_bf16(int lb, const PairArgs& p, hipStream_t s);
hipError_t linear_launch_fp16(int tile, bool direct, int la, int lb, const LinearArgs& g,
                              hipStream_t s);
hipError_t linear_launch_bf16(int tile, bool direct, int la, int lb, const LinearArgs& g,
                              hipStream_t s);

}  // namespace mmaops
#endif
