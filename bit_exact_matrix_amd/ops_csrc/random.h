// random.h -- dropout's mask from a counter, and the dropout of a matrix.
//
// Philox4x32 with ten rounds (Salmon, Moraes, Dror, Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011): a bijection of 128-bit counters
// under a 64-bit key.  One call gives four words, here eight 16-bit numbers:
// those of eight neighbouring elements of a row.  The counter's lower half is
// row * 2^24 + column / 8, its upper half the call's offset, the key its seed,
// so a mask goes by an element's place alone: not by the kernel, the tile or
// the number of rows, and whoever needs it again makes it again.
//
// 16 bits an element: keeping is decided to within 2^-17 of p, and what is
// kept is divided by the share that truly is, (65536 - T) / 65536.  32 bits take two
// calls for eight elements: 8192 x 4096 bf16 33 us, one call 25 (134 MB, 5.4 TB/s, a
// copy's rate); in the forward residual sum 60 and 54.
#ifndef MMAOPS_RANDOM_H
#define MMAOPS_RANDOM_H

#include "norm.h"

namespace mmaops {

struct DropArgs {
  uint64_t seed, offset;
  const uint64_t* state;  // device memory, or NULL: seed and offset in their place
  uint32_t threshold;     // 0 (nothing is dropped) to 65536 (everything)
  float up;               // 65536 / (65536 - threshold), 0 where all is dropped
};

// seed and offset, in scalar registers
struct Drop {
  uint32_t k0, k1, o0, o1, threshold;
  float up;
  __device__ __forceinline__ explicit Drop(const DropArgs& a) {
    const uint64_t seed = a.state && a.threshold ? a.state[0] : a.seed;
    const uint64_t offset = a.state && a.threshold ? a.state[1] : a.offset;
    k0 = __builtin_amdgcn_readfirstlane((uint32_t)seed);
    k1 = __builtin_amdgcn_readfirstlane((uint32_t)(seed >> 32));
    o0 = __builtin_amdgcn_readfirstlane((uint32_t)offset);
    o1 = __builtin_amdgcn_readfirstlane((uint32_t)(offset >> 32));
    threshold = a.threshold;
    up = a.up;
  }

  // The numbers of elements c to c + 7 of a row (c a multiple of 8), two a
  // word, the lower column in the lower half.
  __device__ __forceinline__ void words(int64_t row, int64_t c, uint32_t (&w)[4]) const {
    const uint64_t count = ((uint64_t)row << 24) + (uint64_t)(c >> 3);
    uint32_t x0 = (uint32_t)count, x1 = (uint32_t)(count >> 32), x2 = o0, x3 = o1;
    uint32_t a = k0, b = k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      const uint64_t p0 = (uint64_t)x0 * 0xD2511F53u, p1 = (uint64_t)x2 * 0xCD9E8D57u;
      x0 = (uint32_t)(p1 >> 32) ^ x1 ^ a;
      x2 = (uint32_t)(p0 >> 32) ^ x3 ^ b;
      x1 = (uint32_t)p1;
      x3 = (uint32_t)p0;
      a += 0x9E3779B9u;
      b += 0xBB67AE85u;
    }
    w[0] = x0;
    w[1] = x1;
    w[2] = x2;
    w[3] = x3;
  }

  // The same of V elements from c on, a multiple of V = 4 or 8.
  template <int V>
  __device__ __forceinline__ void halves(int64_t row, int64_t c, uint32_t (&w)[V / 2]) const {
    static_assert(V == 4 || V == 8, "");
    uint32_t q[4];
    words(row, c, q);
    if constexpr (V == 8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = q[i];
    } else {
      w[0] = c & 4 ? q[2] : q[0];
      w[1] = c & 4 ? q[3] : q[1];
    }
  }

  // What is dropped is 0 whatever it was, an infinity or NaN too.
  template <int V>
  __device__ __forceinline__ void apply(const uint32_t (&w)[V / 2], float (&v)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t u = i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu;
      v[i] = u >= threshold ? v[i] * up : 0.0f;
    }
  }

  // 0 where it is dropped, without the factor
  template <int V>
  __device__ __forceinline__ void clear(const uint32_t (&w)[V / 2], float (&v)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t u = i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu;
      v[i] = u >= threshold ? v[i] : 0.0f;
    }
  }
};

// y = drop(x) + residual, each element read and written once, 8 a lane.  A
// workgroup of 256 lanes is cut into rows of 2^shift lanes, as many as a row has
// groups of 8 elements (16 at least), or, with EXACT, for short rows, into rows of
// `lanes` lanes, as many as there are groups: fewer stand idle (bf16, 104857 x 320
// 39 us and 30, 52428 x 640 35 and 31), but the address takes more (8192 x 4096 24.5
// and 28).  inverse: 65536 / lanes + 1, with which a lane's row is found in one
// product, exact below 256.
struct DropGrid {
  int shift, lanes, inverse;
};
template <int DT, bool EXACT>
__global__ __launch_bounds__(256) void dropout_kernel(const void* x, int64_t ldx,
                                                      const void* residual, int64_t ldr, void* y,
                                                      int64_t ldy, int64_t rows, int64_t cols,
                                                      DropArgs args, DropGrid cut) {
  constexpr int V = 8;
  using E = elem_t<DT>;
  const Drop drop(args);
  const int lanes = EXACT ? cut.lanes : 1 << cut.shift;
  const int per = EXACT ? 256 / lanes : 256 >> cut.shift;
  const int g = EXACT ? (int)threadIdx.x * cut.inverse >> 16 : (int)threadIdx.x >> cut.shift;
  const int lane = EXACT ? (int)threadIdx.x - g * lanes : (int)threadIdx.x & (lanes - 1);
  if (EXACT && g >= per) return;
  const int64_t step = (int64_t)gridDim.x * per;
  const int64_t c0 = (int64_t)blockIdx.y * lanes * V, cstep = (int64_t)gridDim.y * lanes * V;
  for (int64_t row = (int64_t)blockIdx.x * per + g; row < rows; row += step)
    for (int64_t c = c0 + lane * V; c < cols; c += cstep) {
      const int n = cols - c < V ? (int)(cols - c) : V;
      float v[V], r[V];
      const Pack<DT, V> px = load_pack<DT, V>((const E*)x + row * ldx + c, n);
      Pack<DT, V> pr;
      if (residual) pr = load_pack<DT, V>((const E*)residual + row * ldr + c, n);
      unpack(px, v);
      if (drop.threshold) {
        uint32_t w[V / 2];
        drop.halves<V>(row, c, w);
        drop.apply<V>(w, v);
      }
      if (residual) {
        unpack(pr, r);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += r[i];
      }
      store_pack<DT, V>((E*)y + row * ldy + c, pack<DT, V>(v), n);
    }
}

}  // namespace mmaops
#endif
