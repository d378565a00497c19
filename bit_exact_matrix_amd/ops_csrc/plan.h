// plan.h -- how a product is run: its tile, the split of its inner size, and
// which operands are copied to aligned rows first.  Host code without HIP, so
// that it can be checked on its own.
#ifndef MMAOPS_PLAN_H
#define MMAOPS_PLAN_H

#include <stdint.h>
#include <stdlib.h>

namespace mmaops {

constexpr int kCUs = 256;

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

// Tile sizes and workgroup shapes (linear.h has the kernels).
enum {
  kTileBig = 0,
  kTileMid = 1,
  kTileSmall = 2,
  kTileFew = 3,
  kTileRows = 4,
  kTileVec = 5,
  kTiles = 6
};
struct TileShape {
  int bm, bn, bk, waves;  // bm, bn: the most rows and columns of a workgroup
  bool pairs;  // a wave holds whole checkpoint blocks
};
constexpr TileShape kTileShape[kTiles] = {
    {256, 256, 64, 4, true},  {128, 128, 64, 4, true}, {64, 64, 64, 4, true},
    {16, 64, 128, 4, false}, {16, 32, 64, 8, true},    {2, 64, 8, 16, true}};

// A product C (M x N) = A B with inner size K, its operands' layouts and
// how it is run.
struct Product {
  int64_t M, N, K;
  int la, lb;
  const void *a, *b;
  int64_t lda, ldb;
};

// direct: direct loads from both operands.  What they cannot be loaded from
// directly is copied to aligned rows first (copy_a, copy_b); for few rows,
// where that reads the weight twice, the tile may go through registers.
struct Plan {
  int tile, splits;
  bool direct, partial, copy_a, copy_b, guard;
};

// MMAOPS_LINEAR_TILE (0 to 5) and MMAOPS_LINEAR_SPLITS: diagnostic
// overrides of the choice below, read on every call, so that each variant
// can be tested on any shape.
inline int env_int(const char* name, int lo, int hi) {
  const char* v = getenv(name);
  if (!v || !*v) return -1;
  char* end = nullptr;
  const long x = strtol(v, &end, 10);
  return end && *end == '\0' && x >= lo && x <= hi ? (int)x : -1;
}

// An estimate of a product's time on one MI355X, in us: `n` workgroups of a
// tile, each `steps` long.  Fitted to times on the GPU from 33 x 4096 x 4096
// to 2048 x 4096 x 4096, 64 x 1024 x 1024 to 8192 x 256 x 1024 and 256 x
// 256 x 65536 (bf16, X W).  What the tiles take there, each side measured:
//   512 x 4096 x 4096    small 31  mid 33  big 77
//   1024 x 4096 x 4096   small 57  mid 35  big 79
//   2048 x 4096 x 4096   small 106 mid 59  big 86
//   4096 x 4096 x 1024             mid 38  big 36
//   64 x 1024 x 1024     few 6.4   small 8.5
//   512 x 512 x 8192     small 36, its inner size split in four 19
inline double tile_time(int tile, int64_t n, int64_t steps) {
  const int64_t full = (n + kCUs - 1) / kCUs;  // workgroups of the fullest CU
  const double even = (double)n / kCUs;
  switch (tile) {
    case kTileBig: return 8.0 + steps * 1.45 * full;
    case kTileMid: return 4.6 + steps * (full / 2 * 0.86 + full % 2 * 0.47);
    case kTileSmall: return 4.6 + steps * (even > 1.3 ? even * 0.2 : 0.26);
    default: return 4.5 + steps * (full > 1 ? full * 0.24 : 0.3);
  }
}

// The tile of few rows through registers: a step waits for its loads, until
// several workgroups share a CU (6 x 2135 x 132, W stored N x K: 33 us in 17
// steps; copied to aligned rows and loaded directly, 12).
inline double few_through_registers_time(int64_t n, int64_t steps) {
  const double even = (double)n / kCUs;
  return 4.5 + steps * (even > 3.6 ? even * 0.5 : 1.8);
}

// an operand of `elements` copied to aligned rows: a launch, read and written
inline double copy_time(int64_t elements) { return 3.0 + (double)elements * 4 / 5e6; }

// the second kernel of a split product: its launch, and the partial sums
// written and read
inline double join_time(int64_t M, int64_t N, int64_t splits) {
  return 4.5 + (double)M * N * splits * 8 / 5e6;
}

// Rows and row length of an operand as it is stored.
struct Stored {
  int64_t rows, cols, ld;  // ld: of its aligned copy
};
inline Stored stored(int layout, int64_t len, int64_t K) {
  const int64_t rows = layout == 0 ? len : K, cols = layout == 0 ? K : len;
  return {rows, cols, (cols + 7) / 8 * 8};
}

// Whether direct loads of a tile reach all of it: their offsets, from the
// tile's first element on, are 32-bit numbers of bytes.  A tile has `most` of
// the operand's `len` rows and `bk` of the inner size.
inline bool in_reach(int layout, int64_t most, int64_t len, int64_t bk, int64_t ld) {
  const int64_t rows = layout == 0 ? (most < len ? most : len) : bk;
  const int64_t row = layout == 0 ? bk : most;
  return rows <= 1 || ld <= ((int64_t(1) << 31) - 1 - row) / (rows - 1);
}

inline Plan linear_plan(const Product& p, bool saves) {
  Plan q;
  // Direct loads take 16-byte pieces of rows that start on 16 bytes.  An
  // operand whose rows do not, or are too far apart for a tile, is copied;
  // rows that are too long even so leave the tile out.
  const bool a16 = aligned(p.a, 16) && p.lda % 8 == 0, b16 = aligned(p.b, 16) && p.ldb % 8 == 0;
  const int64_t copy_lda = stored(p.la, p.M, p.K).ld, copy_ldb = stored(p.lb, p.N, p.K).ld;
  enum Load { kAsItIs, kCopied, kNot };
  auto load_a = [&](int t) {
    const TileShape& s = kTileShape[t];
    return a16 && in_reach(p.la, s.bm, p.M, s.bk, p.lda)  ? kAsItIs
           : in_reach(p.la, s.bm, p.M, s.bk, copy_lda) ? kCopied
                                                       : kNot;
  };
  auto load_b = [&](int t) {
    const TileShape& s = kTileShape[t];
    return b16 && in_reach(p.lb, s.bn, p.N, s.bk, p.ldb)  ? kAsItIs
           : in_reach(p.lb, s.bn, p.N, s.bk, copy_ldb) ? kCopied
                                                       : kNot;
  };
  auto tiles = [&](int t) {
    const TileShape& s = kTileShape[t];
    return ((p.M + s.bm - 1) / s.bm) * ((p.N + s.bn - 1) / s.bn);
  };
  // all of K in one workgroup: whole steps, from direct loads that need no
  // guard, one workgroup for each CU at most, while K is short enough (bf16,
  // weights from memory, rows against few: 1 x 4096 x 4096 W stored N x K
  // 10.5 us and 12.4, K x N 18.9 and 14.0; 1 x 4096 x 1024 4.9 and 5.8, 5.8
  // and 6.2; 1 x 8192 x 4096 19.8 and 18.2; 16 x 512 x 8192 13.1 and 9.7)
  const bool rows_fit = p.M <= 16 && p.la == 0 && a16 && load_b(kTileRows) == kAsItIs &&
                        p.K > 0 && p.K % 64 == 0 && (p.lb == 0 || p.N % 8 == 0);
  // One or two rows against rows of the weight, through registers: where
  // direct loads would need copies of them, while one workgroup for each CU
  // is enough and K is short (1 x 255 x 2047 9.3 us, with copies 16.5; 1 x
  // 16383 x 2047 20.5 and 24.3; but 1 x 1023 x 8191 29.5 and 26.3, 1 x 50001
  // x 128 12.5 and 8.6), but more than the one step that the tile of few rows
  // needs no second launch for (1 x 16383 x 127: 8.0 and 6.6; with z saved it
  // needs one, 8.2 and 9.5, but what is saved does not choose the order of
  // the sums).
  const bool vec_fit =
      p.M <= 2 && p.la == 0 && p.lb == 1 && p.K > 0 && p.N <= (int64_t(1) << 25);
  const int env_tile = env_int("MMAOPS_LINEAR_TILE", 0, kTiles - 1);
  const int env_splits = env_int("MMAOPS_LINEAR_SPLITS", 1, 4096);
  q.tile = kTileFew;
  q.splits = 1;
  q.direct = true;
  q.copy_a = q.copy_b = false;
  const bool few_as_is = load_a(kTileFew) == kAsItIs && load_b(kTileFew) == kAsItIs;
  const bool vec_wins = !few_as_is && p.K <= 2048 && p.K > 128 && p.N <= 64 * kCUs;
  if (vec_fit && (env_tile < 0 ? vec_wins : env_tile == kTileVec)) {
    q.tile = kTileVec;
  } else if (env_tile == kTileRows ? rows_fit
                            : env_tile < 0 && rows_fit && p.N <= 16 * kCUs &&
                                  p.K <= (p.lb == 0 ? 4096 : 1024)) {
    q.tile = kTileRows;
  } else {
    double best = 1e300;
    // Rows too long for the direct loads of every tile considered: the tile
    // of few rows, whose offsets through registers are of 64 bits.
    for (int any = 0; any <= 1 && best == 1e300; ++any)
      for (int v = 0; v <= kTileFew + 1; ++v) {  // the last: few rows through registers
        const int t = v < kTileFew ? v : kTileFew;
        const bool direct = v <= kTileFew;
        if (any                ? t != kTileFew
            : env_tile >= 0    ? t != (env_tile < kTileFew ? env_tile : kTileFew)
            : t == kTileFew    ? p.M > 128
                               : p.M <= 16)
          continue;
        const Load a = load_a(t), b = load_b(t);
        if (direct ? a == kNot || b == kNot : !any && few_as_is) continue;
        const double copies = (a == kCopied ? copy_time(p.M * p.K) : 0.0) +
                              (b == kCopied ? copy_time(p.N * p.K) : 0.0);
        const int64_t steps = (p.K + kTileShape[t].bk - 1) / kTileShape[t].bk, n = tiles(t);
        if (t != kTileBig && t != kTileFew && n * kTileShape[t].waves * 64 > UINT32_MAX)
          continue;  // more lanes than a grid has in x
        for (int s = 1; s <= 32; s += s < 4 ? 1 : s / 2) {
          const int k = env_splits >= 0 ? (int)(env_splits < steps ? env_splits : steps) : s;
          if (env_splits < 0 && s > 1 && steps / s < (direct ? 4 : 1)) break;
          const int64_t run = (steps + s - 1) / s;
          const double time = (direct ? tile_time(t, n * s, run) + copies
                                      : few_through_registers_time(n * s, run)) +
                              (s > 1 ? join_time(p.M, p.N, s) : 0.0);
          if (time < best) {
            best = time;
            q.tile = t;
            q.direct = direct;
            q.copy_a = direct && a == kCopied;
            q.copy_b = direct && b == kCopied;
            q.splits = k < 1 ? 1 : k;
          }
          if (env_splits >= 0) break;
        }
      }
  }
  q.guard = q.direct && ((p.la == 1 && p.M % 8 && !q.copy_a) ||
                         (p.lb == 1 && p.N % 8 && !q.copy_b));
  q.partial = q.splits > 1 || (saves && !kTileShape[q.tile].pairs);
  return q;
}

// What a product takes of the workspace: the partial sums, then the copies.
inline int64_t partial_bytes(const Product& p, const Plan& q) {
  return q.partial ? up256(p.M * p.N * q.splits * 4) : 0;
}
inline int64_t copy_bytes(bool copy, const Stored& t) {
  return copy ? up256(t.rows * t.ld * 2) : 0;
}
inline int64_t product_bytes(const Product& p, const Plan& q) {
  return partial_bytes(p, q) + copy_bytes(q.copy_a, stored(p.la, p.M, p.K)) +
         copy_bytes(q.copy_b, stored(p.lb, p.N, p.K));
}

// ------------------------------------------- products of a gated layer
// kGated  C, C2 (M x N each) = A B, A B2, a tile with the same columns of both
// kSummed C = A B + A2 B2
// kApart  C = A B and C2 = A2 B2, in one launch
// of inner size K each (linear.h and gated.h have the kernels).  Operands of a
// pair have the same layout; where their leading dimensions differ both are
// copied, as where their rows do not start on 16 bytes.
enum { kGated = 0, kSummed = 1, kApart = 2 };
struct Paired {
  int kind;
  Product p;
  const void *a2, *b2;  // a2 NULL: a itself; b2 NULL: b itself
  int64_t lda2, ldb2;
};

// The gated tile of few rows, 37 KB a step, one workgroup a CU at a time.  Up to
// 128 workgroups wait for their loads, from there on they share the memory's rate
// (K = 4096, weights from memory, K whole, split in two, four, eight: 1 x 4096 K x N 36
// us, 25, 21 and 22; 16 x 8192 K x N 40, 35, 34 and 36, N x K 39, 35, 32 and 44; 1 x
// 11008 N x K 44, 46, 40 and 48).
inline double gated_few_time(int layout, int64_t n, int64_t steps) {
  const double even = (double)n / kCUs, full = (double)((n + kCUs - 1) / kCUs);
  const double step = n <= 128    ? 1.05
                      : n <= kCUs ? 1.05 + (n - 128) / 128.0 * 0.45
                                  : (even + full) / 2 * (layout == 0 ? 1.35 : 1.5);
  return 4.5 + steps * step;
}

// The most columns of a tile's right operands, each (for few rows the gated
// tile is twice as wide as a plain one).
inline int paired_columns(int kind, int tile) {
  if (kind != kGated || tile == kTileRows) return kTileShape[tile].bn;
  return tile == kTileFew ? 64 : kTileShape[tile].bn / 2;
}

inline Plan paired_plan(const Paired& q, bool saves) {
  const Product& p = q.p;
  Plan r;
  // a kernel has one leading dimension for both of a pair
  const bool apart_a = q.a2 && q.lda2 != p.lda, apart_b = q.b2 && q.ldb2 != p.ldb;
  const bool a16 = !apart_a && aligned(p.a, 16) && p.lda % 8 == 0 && aligned(q.a2, 16);
  const bool b16 = !apart_b && aligned(p.b, 16) && p.ldb % 8 == 0 && aligned(q.b2, 16);
  const Stored sa = stored(p.la, p.M, p.K), sb = stored(p.lb, p.N, p.K);
  enum Load { kAsItIs, kCopied, kNot };
  auto load_a = [&](int t) {
    const TileShape& s = kTileShape[t];
    return a16 && in_reach(p.la, s.bm, p.M, s.bk, p.lda) ? kAsItIs
           : in_reach(p.la, s.bm, p.M, s.bk, sa.ld)      ? kCopied
                                                         : kNot;
  };
  auto load_b = [&](int t) {
    const int64_t most = paired_columns(q.kind, t), bk = kTileShape[t].bk;
    return b16 && in_reach(p.lb, most, p.N, bk, p.ldb) ? kAsItIs
           : in_reach(p.lb, most, p.N, bk, sb.ld)      ? kCopied
                                                       : kNot;
  };
  // what one tile's product takes twice
  const int64_t times = q.kind == kApart ? 2 : 1, parts = q.kind == kSummed ? 2 : 1;
  const int64_t sums = q.kind == kSummed ? 1 : 2;  // FP32 sums of an output place
  const int env_tile = env_int("MMAOPS_LINEAR_TILE", 0, kTiles - 1);
  const int env_splits = env_int("MMAOPS_LINEAR_SPLITS", 1, 4096);
  const bool few_as_is = load_a(kTileFew) == kAsItIs && load_b(kTileFew) == kAsItIs;
  r.tile = kTileFew;
  r.splits = 1;
  r.direct = false;
  r.copy_a = r.copy_b = false;
  double best = 1e300;
  // All of K in one workgroup of 16 columns of both, by the rule of a plain
  // product (weights from memory, rows against few: 1 x 4096 x 4096 N x K 16.2 us
  // and 17.4, K x N 31.5 and 21.3; 16 x 4096 x 1024 6.1 and 7.3, 8.1 and 8.7; 16 x
  // 8192 x 4096 N x K 33.2 and 31.6).
  const bool rows_fit = q.kind == kGated && p.M <= 16 && a16 && load_b(kTileRows) == kAsItIs &&
                        p.K > 0 && p.K % 64 == 0 && (p.lb == 0 || p.N % 8 == 0);
  const bool rows_win = p.N <= 16 * kCUs && p.K <= (p.lb == 0 ? 4096 : 1024);
  if (rows_fit && (env_tile < 0 ? rows_win : env_tile == kTileRows)) {
    r.tile = kTileRows;
    r.direct = true;
    best = 0.0;
  }
  for (int any = 0; any <= 1 && best == 1e300; ++any)
    for (int v = 0; v <= kTileFew + 1; ++v) {  // the last: few rows through registers
      const int t = v < kTileFew ? v : kTileFew;
      const bool direct = v <= kTileFew;
      if (any                ? t != kTileFew
          : env_tile >= 0    ? t != (env_tile < kTileFew ? env_tile : kTileFew)
          : t == kTileFew    ? p.M > 128
                             : p.M <= 16)
        continue;
      const Load a = load_a(t), b = load_b(t);
      if (direct ? a == kNot || b == kNot : !any && few_as_is) continue;
      const bool copy_a = direct ? a == kCopied : apart_a;
      const bool copy_b = direct ? b == kCopied : apart_b;
      const double copies = (copy_a ? copy_time(p.M * p.K * (q.a2 ? 2 : 1)) : 0.0) +
                            (copy_b ? copy_time(p.N * p.K * (q.b2 ? 2 : 1)) : 0.0);
      const int64_t cols = paired_columns(q.kind, t), bk = kTileShape[t].bk;
      const int64_t steps = (p.K + bk - 1) / bk * parts;
      const int64_t n = (p.M + kTileShape[t].bm - 1) / kTileShape[t].bm * ((p.N + cols - 1) / cols);
      for (int s = 1; s <= 32; s += s < 4 ? 1 : s / 2) {
        const int k = env_splits >= 0 ? (int)(env_splits < steps ? env_splits : steps) : s;
        if (env_splits < 0 && s > 1 && steps / s < (direct ? 4 : 1)) break;
        const int64_t run = (steps + s - 1) / s;
        const double time = (!direct ? few_through_registers_time(n * s * times, run)
                             : q.kind == kGated && t == kTileFew
                                 ? gated_few_time(p.lb, n * s, run)
                                 : tile_time(t, n * s * times, run)) +
                            copies + (s > 1 ? join_time(p.M, p.N * sums, s) : 0.0);
        if (time < best) {
          best = time;
          r.tile = t;
          r.direct = direct;
          r.copy_a = copy_a;
          r.copy_b = copy_b;
          r.splits = k < 1 ? 1 : k;
        }
        if (env_splits >= 0) break;
      }
    }
  r.guard = r.direct && ((p.la == 1 && p.M % 8 && !r.copy_a) ||
                         (p.lb == 1 && p.N % 8 && !r.copy_b));
  // a wave of the gated 64 x 64 tile has 16 columns of each, half a block
  r.partial = r.splits > 1 || (saves && (r.tile == kTileSmall || r.tile == kTileFew));
  return r;
}

// What it takes of the workspace: the partial sums, then the copies.
inline int64_t paired_partial_bytes(const Paired& q, const Plan& r) {
  return r.partial ? up256(q.p.M * q.p.N * r.splits * 4 * (q.kind == kSummed ? 1 : 2)) : 0;
}
inline int64_t paired_bytes(const Paired& q, const Plan& r) {
  return paired_partial_bytes(q, r) +
         copy_bytes(r.copy_a, stored(q.p.la, q.p.M, q.p.K)) * (q.a2 ? 2 : 1) +
         copy_bytes(r.copy_b, stored(q.p.lb, q.p.N, q.p.K)) * (q.b2 ? 2 : 1);
}

}  // namespace mmaops
#endif
