// Element types, gates and 8-bit codes shared by the gated-scan and checkpoint kernels.
#pragma once

#include "gated_internal.h"

namespace ssdq {

template <typename T>
__device__ __forceinline__ float to_f32(T v) { return float(v); }
// The binary32 value rounded to nearest even.  The value is made opaque first: the compiler would
// else fuse the operation that forms it with the conversion to binary16 in some kernels and not in
// others (one rounding instead of two), and the same h would have two images.
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  if constexpr (__is_same(T, _Float16)) asm("" : "+v"(v));
  return T(v);
}

// exp(x).  -inf gives 0, +inf gives +inf, a result below 2^-126 gives 0.
//
// EXACT (for binary32 tensors): within 3 * 2^-24 of itself, the product x log2(e) carried as a pair whose low part
// is applied to the hardware exp2 as a factor 1 + low ln 2.  Otherwise exp2 of the rounded product, within
// (|x| + 2) 2^-24: for tensors of 16 bits that vanishes in their rounding, and in a state the part with |x|
// cannot add up, since a gate of log x is forgotten after about 1 / |x| tokens.
template <bool EXACT>
__device__ __forceinline__ float exp_f32(float x) {
  constexpr float kLog2e = 1.44269502e+00f;      // log2(e) rounded to binary32
  constexpr float kLog2eLow = 1.92596298e-08f;   // log2(e) - kLog2e
  constexpr float kLn2 = 6.93147182e-01f;
  const float hi = x * kLog2e;
  const float e = __builtin_amdgcn_exp2f(hi);
  if constexpr (!EXACT) return e;
  const float lo = fmaf(x, kLog2eLow, fmaf(x, kLog2e, -hi));
  // overflow, underflow, infinities and NaN: e alone is the answer (lo may be NaN there)
  return fabsf(hi) < 128.f ? fmaf(e, lo * kLn2, e) : e;
}

// A logit's two sigmoids, a and 1 - a, as one number: the smaller of them (which keeps its relative precision), with
// the logit's sign.
template <bool EXACT>
__device__ __forceinline__ float logit_pair(float g) {
  const float e = exp_f32<EXACT>(-fabsf(g)), sum = 1.f + e;
  float inv = __builtin_amdgcn_rcpf(sum);
  // The hardware reciprocal is within 1.6 of 2^-24 and low by 0.1 of it on average.  For binary32 tensors one Newton
  // step follows; beside the rounding of 16-bit ones it is not seen: the smaller sigmoid is low by 6e-9 of itself, and the
  // other one, 1 - that, high by as many parts of the smaller.  A state of memory 1 / (1 - a), which adds (1 - a) u, is
  // moved by less than 6e-9 of the magnitudes in it, however long it is.
  if constexpr (EXACT) inv = fmaf(fmaf(-sum, inv, 1.f), inv, inv);
  return copysignf(e * inv, g);
}
__device__ __forceinline__ void split_pair(float pair, float& a, float& c) {
  const float low = fabsf(pair), high = 1.f - low;
  const bool negative = __float_as_int(pair) < 0;
  a = negative ? low : high;
  c = negative ? high : low;
}

// The gate's a, and what multiplies u in b (1 for a log gate).
template <int KIND, bool EXACT>
__device__ __forceinline__ void gate_terms(float g, float& a, float& c) {
  if constexpr (KIND == SSDQ_GATE_LOG) {
    a = exp_f32<EXACT>(g);
    c = 1.f;
  } else {
    split_pair(logit_pair<EXACT>(g), a, c);
  }
}

// 8-bit codes of a block whose largest magnitude m has the binary32 image `most`: the scale, m
// times the binary32 1/127 (0 below the normal range, NaN for a block that is not finite).
__device__ __forceinline__ float checkpoint_scale(uint32_t most) {
  if (most >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  const float m = __uint_as_float(most);
  constexpr float kSmallest = 127.f * 1.17549435e-38f;   // 127 * 2^-126
  return m < kSmallest ? 0.f : m * (1.f / 127.f);
}

typedef unsigned short u16;

// An unsigned word, or vector of words, of VB bytes
template <int VB>
struct Bytes;
template <>
struct Bytes<16> { typedef v4u type; };
template <>
struct Bytes<8> { typedef v2u type; };
template <>
struct Bytes<4> { typedef uint32_t type; };
template <>
struct Bytes<2> { typedef u16 type; };
template <>
struct Bytes<1> { typedef uint8_t type; };
struct Halves { v4u h[2]; };

// V neighbouring elements as loaded
template <typename T, int V>
struct Pack {
  typedef typename Bytes<sizeof(T) * V>::type Raw;
  struct Elements { T e[V]; };
  Raw raw;
  __device__ __forceinline__ float operator[](int v) const { return to_f32(__builtin_bit_cast(Elements, raw).e[v]); }
};
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> to_pack(const float (&x)[V]) {
  typename Pack<T, V>::Elements e;
#pragma unroll
  for (int v = 0; v < V; ++v) e.e[v] = from_f32<T>(x[v]);
  return Pack<T, V>{__builtin_bit_cast(typename Pack<T, V>::Raw, e)};
}

// The codes of V neighbouring elements under scale s, packed: the integers nearest to the exact quotients, ties
// to even.  k = rint(v rcp(s)), formed in the binade of 1.5 * 2^23 where the spacing is 1, is one of the two
// nearest integers (the product is within 2^-14 of the quotient), and r = v - k s is exact in one fma (it stays
// near s / 2 and is a multiple of the smaller operand's last place).  So k is right wherever |r| < s / 2, and
// only where some |r| of the V reaches it does a branch decide.  A zero or NaN scale codes everything as 0.
template <int V, typename P>
__device__ __forceinline__ typename Bytes<V>::type codes_of(const P& x, float s) {
  constexpr float kRound = 12582912.f;   // 1.5 * 2^23
  struct { int8_t e[V]; } q = {};
  if (s > 0.f) {
    const float rcp = __builtin_amdgcn_rcpf(s), half = 0.5f * s;
    float t[V], r[V], most = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      t[v] = fmaf(x[v], rcp, kRound);
      r[v] = fmaf(-(t[v] - kRound), s, x[v]);
      most = fmaxf(most, fabsf(r[v]));
    }
    if (most >= half) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const bool odd = __float_as_uint(t[v]) & 1u;
        if (fabsf(r[v]) > half || (fabsf(r[v]) == half && odd)) t[v] += r[v] > 0.f ? 1.f : -1.f;
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) q.e[v] = int8_t(__float_as_uint(t[v]) & 0xffu);   // the integer's low byte
  }
  return __builtin_bit_cast(typename Bytes<V>::type, q);
}

// The largest magnitude of the first `count` of V elements, as the image of a binary32 number: magnitudes compare
// as integers, NaN above infinity above the rest.
typedef unsigned short v2us __attribute__((ext_vector_type(2)));
template <typename T, int V>
__device__ __forceinline__ uint32_t largest(const Pack<T, V>& x, int count) {
  if constexpr (sizeof(T) == 2 && V == 8) {
    v4u w = x.raw & 0x7fff7fffu;
    if (count < V) {   // the elements past the row's end count as 0
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] &= 2 * k + 1 < count ? 0xffffffffu : 2 * k < count ? 0xffffu : 0u;
    }
    const uint32_t w0 = w[0], w1 = w[1], w2 = w[2], w3 = w[3];
    const v2us m = __builtin_elementwise_max(
        __builtin_elementwise_max(__builtin_bit_cast(v2us, w0), __builtin_bit_cast(v2us, w1)),
        __builtin_elementwise_max(__builtin_bit_cast(v2us, w2), __builtin_bit_cast(v2us, w3)));
    const unsigned short top = m[0] > m[1] ? m[0] : m[1];
    return __float_as_uint(to_f32(__builtin_bit_cast(T, top)));
  } else {
    uint32_t most = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v < count) most = max(most, __float_as_uint(fabsf(x[v])));
    return most;
  }
}

// Largest of the unsigned images over the lanes of a row's 64 channels (LPR consecutive lanes), in
// every one of them: magnitudes compare as integers, NaN above infinity above the rest.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_umax(uint32_t v) {
  return max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xF, 0xF, false)));
}
template <int LPR>
__device__ __forceinline__ uint32_t row_umax(uint32_t m) {
  if constexpr (LPR >= 2) m = dpp_umax<0xB1>(m);
  if constexpr (LPR >= 4) m = dpp_umax<0x4E>(m);
  if constexpr (LPR >= 8) m = dpp_umax<0x141>(m);
  if constexpr (LPR >= 16) m = dpp_umax<0x140>(m);
  if constexpr (LPR >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    m = max(uint32_t(r[0]), uint32_t(r[1]));
  }
  if constexpr (LPR >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    m = max(uint32_t(r[0]), uint32_t(r[1]));
  }
  return m;
}

}  // namespace ssdq
