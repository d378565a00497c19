// ops_common.h -- what the native operators share: element types, vector
// loads, reductions, activations and the 8-bit checkpoint format.  The
// operators themselves are stated in include/mmaops.h.
#ifndef MMAOPS_COMMON_H
#define MMAOPS_COMMON_H

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mmaops {

// element types: the values of include/mmaops.h
constexpr int kFP16 = 0, kBF16 = 1, kFP32 = 3;

using half8 = __attribute__((ext_vector_type(8))) _Float16;
using bf8 = __attribute__((ext_vector_type(8))) __bf16;
using half4 = __attribute__((ext_vector_type(4))) _Float16;
using f32x4 = __attribute__((ext_vector_type(4))) float;
using u32x4 = __attribute__((ext_vector_type(4))) uint32_t;
using u32x2 = __attribute__((ext_vector_type(2))) uint32_t;

template <int DT>
struct Elem;
template <>
struct Elem<kFP16> {
  using type = _Float16;
};
template <>
struct Elem<kBF16> {
  using type = __bf16;
};
template <>
struct Elem<kFP32> {
  using type = float;
};
template <int DT>
using elem_t = typename Elem<DT>::type;

__host__ __device__ constexpr int elem_bytes(int dt) { return dt == kFP32 ? 4 : 2; }

// One element of a type known at run time (a wave-uniform branch).
__device__ __forceinline__ float load_any(const void* p, int64_t i, int dt) {
  if (dt == kFP32) return ((const float*)p)[i];
  if (dt == kFP16) return (float)((const _Float16*)p)[i];
  return (float)((const __bf16*)p)[i];
}

__device__ __forceinline__ void store_any(void* p, int64_t i, float v, int dt) {
  if (dt == kFP32)
    ((float*)p)[i] = v;
  else if (dt == kFP16)
    ((_Float16*)p)[i] = (_Float16)v;
  else
    ((__bf16*)p)[i] = (__bf16)v;
}

// V consecutive elements, in registers as they are in memory, word by word
// (element by element the compiler would give each 16-bit one a register).
// Global loads and stores of 16 bytes need no more than the element's
// alignment on gfx950, so rows of odd lengths and strides take the same
// wide accesses.
template <int DT, int V>
struct Pack {
  static constexpr int kWords = V * elem_bytes(DT) / 4;
  uint32_t w[kWords];
};

template <int DT, int V>
__device__ __forceinline__ Pack<DT, V> load_pack(const elem_t<DT>* p) {
  Pack<DT, V> q;
  __builtin_memcpy(q.w, p, sizeof q.w);
  return q;
}

// The first `bytes` (fewer than 4 W; a multiple of UNIT) of W words, 0 for
// the others: one access for each power of two in it, all on their way
// before the first is used (element by element they waited for each other:
// layer norm 8192 x 4095 bf16 with checkpoint 48 us, so 44, backward 72 and
// 61).
template <int W, int UNIT>
__device__ __forceinline__ void load_part(const void* p, int bytes, uint32_t (&w)[W]) {
  static_assert(W <= 4, "powers of two below 16 bytes");
  const char* const c = (const char*)p;
  uint32_t a[2] = {0, 0}, b = 0;
  uint16_t h = 0;
  uint8_t o = 0;
  if (W > 2 && (bytes & 8)) __builtin_memcpy(a, c, 8);
  if (W > 1 && (bytes & 4)) __builtin_memcpy(&b, c + (bytes & 8), 4);
  if (UNIT < 4 && (bytes & 2)) __builtin_memcpy(&h, c + (bytes & 12), 2);
  if (UNIT < 2 && (bytes & 1)) o = *(const uint8_t*)(c + (bytes & 14));
#pragma unroll
  for (int i = 0; i < W; ++i) {
    uint32_t v = 0;
    if (W > 2 && i < 2 && (bytes & 8)) v = a[i];
    if (W > 1 && (bytes & 4) && i == (bytes & 8) / 4) v = b;
    if (UNIT < 4 && (bytes & 2) && i == (bytes & 12) / 4) v |= h;
    if (UNIT < 2 && (bytes & 1) && i == (bytes & 14) / 4) v |= (uint32_t)o << (8 * (bytes & 2));
    w[i] = v;
  }
}

// the first n (0 to V) of them; the others are 0
template <int DT, int V>
__device__ __forceinline__ Pack<DT, V> load_pack(const elem_t<DT>* p, int n) {
  if constexpr (Pack<DT, V>::kWords > 4) {
    Pack<DT, V> q;
    const Pack<DT, V / 2> lo = load_pack<DT, V / 2>(p, n);
    const Pack<DT, V / 2> hi = load_pack<DT, V / 2>(p + V / 2, n - V / 2);
#pragma unroll
    for (int i = 0; i < Pack<DT, V / 2>::kWords; ++i) {
      q.w[i] = lo.w[i];
      q.w[Pack<DT, V / 2>::kWords + i] = hi.w[i];
    }
    return q;
  } else {
    if (n >= V) return load_pack<DT, V>(p);
    Pack<DT, V> q;
    if (n <= 0) {
#pragma unroll
      for (int i = 0; i < Pack<DT, V>::kWords; ++i) q.w[i] = 0;
      return q;
    }
    load_part<Pack<DT, V>::kWords, elem_bytes(DT)>(p, n * elem_bytes(DT), q.w);
    return q;
  }
}

template <int DT, int V>
__device__ __forceinline__ void store_pack(elem_t<DT>* p, const Pack<DT, V>& q, int n) {
  if (n >= V) {
    __builtin_memcpy(p, q.w, sizeof q.w);
    return;
  }
  // element by element: stores are not waited for, and in larger parts
  // they shared code with the whole store and split that
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (i >= n) continue;
    if constexpr (DT == kFP32)
      ((uint32_t*)p)[i] = q.w[i];
    else
      ((uint16_t*)p)[i] = (uint16_t)(q.w[i / 2] >> (16 * (i & 1)));
  }
}

template <int DT, int V>
__device__ __forceinline__ void unpack(const Pack<DT, V>& q, float (&v)[V]) {
  if constexpr (DT == kFP32) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = __uint_as_float(q.w[i]);
  } else if constexpr (DT == kBF16) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      v[i] = __uint_as_float(q.w[i / 2] << 16);
      v[i + 1] = __uint_as_float(q.w[i / 2] & 0xFFFF0000u);
    }
  } else {
    using h2 = __attribute__((ext_vector_type(2))) _Float16;
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const h2 h = __builtin_bit_cast(h2, q.w[i / 2]);
      v[i] = (float)h[0];
      v[i + 1] = (float)h[1];
    }
  }
}

template <int DT, int V>
__device__ __forceinline__ Pack<DT, V> pack(const float (&v)[V]) {
  Pack<DT, V> q;
  if constexpr (DT == kFP32) {
#pragma unroll
    for (int i = 0; i < V; ++i) q.w[i] = __float_as_uint(v[i]);
  } else {
    using f2 = __attribute__((ext_vector_type(2))) float;
    using e2 = __attribute__((ext_vector_type(2))) elem_t<DT>;
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const e2 h = __builtin_convertvector((f2){v[i], v[i + 1]}, e2);
      q.w[i / 2] = __builtin_bit_cast(uint32_t, h);
    }
  }
  return q;
}

// ---------------------------------------------------------- reductions
// Lane exchanges without LDS: the value of another lane of the 16-lane row
// (CTRL: quad_perm, row_ror or row_half_mirror).
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141;
constexpr int kRor2 = 0x122, kRor4 = 0x124, kRor8 = 0x128;

// Sum over the 64 lanes of a wave, the same bits in every lane: each step
// adds two values that both lanes of a pair hold.
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<kXor1>(v);
  v += dpp<kXor2>(v);
  v += dpp<kRor8>(v);  // a quad's lanes are equal: quads k and k + 2, then all
  v += dpp<kRor4>(v);
  // rows 0 and 1, 2 and 3; then the halves
  auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// a's sums in the lower half and b's in the upper, over the two halves; the
// same for even and odd rows of 16 lanes.
__device__ __forceinline__ float swap_add32(float a, float b) {
  const auto p =
      __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}
__device__ __forceinline__ float swap_add16(float a, float b) {
  const auto p =
      __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// Sum of V values (a power of two) in pairs: a third of the roundings on
// each value's way that a chain has.
template <int V>
__device__ __forceinline__ float pair_sum(const float (&v)[V]) {
  float t[V];
#pragma unroll
  for (int i = 0; i < V; ++i) t[i] = v[i];
#pragma unroll
  for (int n = V / 2; n > 0; n /= 2)
#pragma unroll
    for (int i = 0; i < n; ++i) t[i] += t[i + n];
  return t[0];
}

// Maximum over 4 or 8 neighbouring lanes.
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  static_assert(LANES == 4 || LANES == 8, "");
  auto with = [&](uint32_t u) { v = u > v ? u : v; };
  with(__float_as_uint(dpp<kXor1>(__uint_as_float(v))));
  with(__float_as_uint(dpp<kXor2>(__uint_as_float(v))));
  if constexpr (LANES == 8) with(__float_as_uint(dpp<kHalfMirror>(__uint_as_float(v))));
  return v;
}

// ---------------------------------------------------------- activations
enum { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

// An epilogue of 256 x 256 outputs on one CU takes 0.43 us for every VALU
// instruction an element, so the functions are written for few of them:
// hardware exp2 and reciprocal (1 ulp each) and no branches.
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kSqrt2OverPi = 0.79788456080286536f;

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float fast_rcp(float x) { return __builtin_amdgcn_rcpf(x); }

__device__ __forceinline__ float logistic(float z) {
  return fast_rcp(1.0f + fast_exp2(-kLog2e * z));
}

// The normal distribution's upper tail, 1 - Phi(a) for a in [0, 13], as 2 to
// the power of its logarithm: a polynomial in a, whose coefficients are a
// least-maximum fit made for this (iteratively reweighted least squares over
// Chebyshev nodes), off by at most 0.6 * 2^-24 log2 of the tail.  The exponent
// is rounded to FP32, so the tail's relative error grows as a^2 / 2: 3e-7 up to
// a = 1, 1e-6 at 3.  (A rational form within 1.5e-7 of 1 had 9e-7 and 5e-5,
// which a float32 output shows; it took 2 us less of 114 in the epilogue at
// 4096^3, and as much less of 244 in that product's backward pass.)  Past 13 the
// tail is below FP32's normal numbers: 0.
constexpr float kTailEnd = 13.0f;

__device__ __forceinline__ float normal_tail(float a) {
  float p = -1.22126891e-13f;
  p = __builtin_fmaf(p, a, 1.12678018e-11f);
  p = __builtin_fmaf(p, a, -4.67293648e-10f);
  p = __builtin_fmaf(p, a, 1.15087335e-08f);
  p = __builtin_fmaf(p, a, -1.87218447e-07f);
  p = __builtin_fmaf(p, a, 2.11248152e-06f);
  p = __builtin_fmaf(p, a, -1.67941016e-05f);
  p = __builtin_fmaf(p, a, 9.18155638e-05f);
  p = __builtin_fmaf(p, a, -0.000298374915f);
  p = __builtin_fmaf(p, a, -4.74745275e-06f);
  p = __builtin_fmaf(p, a, 0.00698830979f);
  p = __builtin_fmaf(p, a, -0.0524861142f);
  p = __builtin_fmaf(p, a, -0.4592022f);
  p = __builtin_fmaf(p, a, -1.15110672f);
  p = __builtin_fmaf(p, a, -0.99999994f);
  return fast_exp2(p);
}

__device__ __forceinline__ float act_apply(float z, int act) {
  switch (act) {
    case kActRelu: return z < 0.0f ? 0.0f : z;  // keeps NaN
    case kActGelu: {
      // z Phi(z) = max(z, 0) - |z| (1 - Phi(|z|)): no cancellation in the
      // lower tail.  The bound keeps an infinity from meeting the zero it
      // makes; NaN comes through the first term.
      const float a = __builtin_amdgcn_fmed3f(__builtin_fabsf(z), 0.0f, kTailEnd);
      return __builtin_fmaf(-a, normal_tail(a), z < 0.0f ? 0.0f : z);
    }
    case kActGeluTanh:
      // (1 + tanh(u)) / 2 = logistic(2u)
      return z * logistic(2.0f * kSqrt2OverPi * z * __builtin_fmaf(0.044715f * z, z, 1.0f));
    case kActSilu: return z * logistic(z);
    default: return z;
  }
}

// z within [-top, top], where what it is multiplied with is 0 beyond: an
// infinity (a pre-activation past its 16-bit type's range) must not become
// NaN there.  NaN comes through the other factor.
__device__ __forceinline__ float bounded(float z, float top) {
  return __builtin_amdgcn_fmed3f(z, -top, top);
}

// d act / d z
__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case kActRelu: return z > 0.0f ? 1.0f : 0.0f;
    case kActGelu: {
      const float b = bounded(z, kTailEnd), q = normal_tail(__builtin_fabsf(b));
      const float e = fast_exp2(z * z * (-0.5f * kLog2e));
      return __builtin_fmaf(b * e, kInvSqrt2Pi, z > 0.0f ? 1.0f - q : q);
    }
    case kActGeluTanh: {
      // 0 or 1 beyond 12, where the product of a zero and a large power
      // of z must not become NaN
      z = z > 12.0f ? 12.0f : z < -12.0f ? -12.0f : z;
      const float z2 = z * z;
      const float s = logistic(2.0f * kSqrt2OverPi * z * __builtin_fmaf(0.044715f, z2, 1.0f));
      return s + z * s * (1.0f - s) * 2.0f * kSqrt2OverPi * (1.0f + 3.0f * 0.044715f * z2);
    }
    case kActSilu: {
      const float s = logistic(z);
      return s * (1.0f + bounded(z, 100.0f) * (1.0f - s));
    }
    default: return 1.0f;
  }
}

// FN of V values, one branch for all of them
template <int V, typename FN>
__device__ __forceinline__ void act_all(float (&v)[V], int act, FN fn) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = fn(v[i], kActRelu);
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = fn(v[i], kActGelu);
      break;
    case kActGeluTanh:
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = fn(v[i], kActGeluTanh);
      break;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = fn(v[i], kActSilu);
      break;
    default:
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = fn(v[i], kActNone);
  }
}

// -------------------------------------------------- 8-bit checkpoints
// E4M3 codes with one power of two for each block of 32 elements of a row.
// A power of two makes x / s exact, so the only rounding is the one to
// E4M3 (nearest, ties to even), and a restored value is exact in the
// element type that was saved: the codes do not depend on the order or
// precision of anything computed here.
constexpr int kBlock = 32;

// The largest magnitude that a checkpoint keeps, so that a code never
// restores to an infinity of the element type: 1.875 times its largest
// power of two (61440 for FP16).
__device__ __forceinline__ constexpr uint32_t save_limit(int dt) {  // FP32 bits
  return dt == kFP16 ? 0x47700000u : 0x7F700000u;
}

// The scale's exponent + 127 from the block's largest magnitude: the
// smallest e with amax <= 448 * 2^e = 1.75 * 2^(e+8).  Adding 0x1FFFFF to
// the pattern carries into the exponent exactly when the fraction is above
// .75.  e is at least -117, where 448 * 2^e still covers every smaller
// block and 2^-9 * 2^e, the smallest value, is a normal BF16 number.
__device__ __forceinline__ int save_scale(uint32_t amax) {  // FP32 bits
  const int e = (int)((amax + 0x1FFFFFu) >> 23) - 127 - 8;
  return (e < -117 ? -117 : e) + 127;
}

// 2^(s - 127), 2^(127 - s) for s in [10, 247]
__device__ __forceinline__ float scale_up(int s) { return __uint_as_float((uint32_t)s << 23); }
__device__ __forceinline__ float scale_down(int s) {
  return __uint_as_float((uint32_t)(254 - s) << 23);
}

// Four E4M3 codes of four scaled values (|v| <= 448 or NaN).
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  return (uint32_t)r;
}

__device__ __forceinline__ void decode4(uint32_t w, float (&v)[4]) {
  v[0] = __builtin_amdgcn_cvt_f32_fp8((int)w, 0);
  v[1] = __builtin_amdgcn_cvt_f32_fp8((int)w, 1);
  v[2] = __builtin_amdgcn_cvt_f32_fp8((int)w, 2);
  v[3] = __builtin_amdgcn_cvt_f32_fp8((int)w, 3);
}

// V codes (4 or 8) as they are in memory, and the first n of them.
template <int V>
struct Codes {
  uint32_t w[V / 4];
};

template <int V>
__device__ __forceinline__ Codes<V> load_codes(const uint8_t* p, int n) {
  Codes<V> c;
  if (n >= V) {
    __builtin_memcpy(&c, p, V);
  } else if (n > 0) {
    load_part<V / 4, 1>(p, n, c.w);
  } else {
#pragma unroll
    for (int j = 0; j < V / 4; ++j) c.w[j] = 0;
  }
  return c;
}

template <int V>
__device__ __forceinline__ void store_codes(uint8_t* p, const Codes<V>& c, int n) {
  if (n >= V) {
    __builtin_memcpy(p, &c, V);
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i < n) p[i] = (uint8_t)(c.w[i / 4] >> (8 * (i & 3)));
}

template <int V>
__device__ __forceinline__ void decode(const Codes<V>& c, int scale, float (&v)[V]) {
  const float up = scale_up(scale);
#pragma unroll
  for (int j = 0; j < V / 4; ++j) {
    float t[4];
    decode4(c.w[j], t);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * j + i] = t[i] * up;
  }
}

// The codes of V consecutive elements held by each lane, where 32 / V
// neighbouring lanes hold a block, from the lane's largest magnitude pattern
// (FP32 bits of |v|).  Elements from n on are not the block's: what they hold
// (a product's tile has sums there) does not count.  Returns the block's
// scale, the same in its lanes.
template <int DT, int V>
__device__ __forceinline__ int encode_with(float (&v)[V], uint32_t mag, int n, Codes<V>& c) {
  constexpr uint32_t limit = save_limit(DT);
  mag = lanes_max<kBlock / V>(mag);
  if (mag > limit) {
    // past the limit, infinities and NaN (a pattern above all others):
    // numbers go to the limit, what is not finite to NaN (E4M3 has no
    // infinity, and an overflow must not come back as a number) and out
    // of the maximum
    mag = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t u = __float_as_uint(v[i]), m = u & 0x7FFFFFFFu;
      const uint32_t t = m < 0x7F800000u ? (m < limit ? m : limit) : 0u;
      mag = t > mag && i < n ? t : mag;
      v[i] = __uint_as_float(m < 0x7F800000u ? (u & 0x80000000u) | t : 0x7FC00000u);
    }
    mag = lanes_max<kBlock / V>(mag);
  }
  const int s = save_scale(mag);
  const float down = scale_down(s);
#pragma unroll
  for (int j = 0; j < V / 4; ++j)
    c.w[j] = encode4(v[4 * j] * down, v[4 * j + 1] * down, v[4 * j + 2] * down,
                     v[4 * j + 3] * down);
  return s;
}

// of FP32 values, saved as the element type DT; those past n do not count
template <int DT, int V>
__device__ __forceinline__ int encode(float (&v)[V], int n, Codes<V>& c) {
  uint32_t mag = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t m = i < n ? __float_as_uint(v[i]) & 0x7FFFFFFFu : 0u;
    mag = m > mag ? m : mag;
  }
  return encode_with<DT, V>(v, mag, n, c);
}

// of elements as they are in memory (0 where there are none)
template <int DT, int V>
__device__ __forceinline__ int encode(const Pack<DT, V>& q, Codes<V>& c) {
  uint32_t mag = 0;
  if constexpr (DT == kFP32) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t m = q.w[i] & 0x7FFFFFFFu;
      mag = m > mag ? m : mag;
    }
  } else {  // two patterns a word
    using u2 = __attribute__((ext_vector_type(2))) uint16_t;
    u2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u2, q.w[i] & 0x7FFF7FFFu));
    const uint16_t top = m[0] > m[1] ? m[0] : m[1];
    mag = DT == kBF16 ? (uint32_t)top << 16
                      : __float_as_uint((float)__builtin_bit_cast(_Float16, top));
  }
  float v[V];
  unpack(q, v);
  return encode_with<DT, V>(v, mag, V, c);
}

}  // namespace mmaops
#endif
