// Element types, gates and 8-bit codes shared by the gated-scan and checkpoint kernels.
#pragma once

#include "ssdq_internal.h"

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

// exp(x) within about 1.5 ulp: the product x log2(e) carried as a pair, its low part applied to
// the hardware exp2 as a factor 1 + lo ln 2.  (The hardware exp2 of the rounded product alone is
// off by |x| 2^-24, which a recurrence over hundreds of tokens would add up.)  -inf gives 0, +inf
// gives +inf, a result below 2^-126 gives 0.
__device__ __forceinline__ float exp_f32(float x) {
  constexpr float kLog2e = 1.44269502e+00f;      // log2(e) rounded to binary32
  constexpr float kLog2eLow = 1.92596298e-08f;   // log2(e) - kLog2e
  constexpr float kLn2 = 6.93147182e-01f;
  const float hi = x * kLog2e;
  const float lo = fmaf(x, kLog2eLow, fmaf(x, kLog2e, -hi));
  const float e = __builtin_amdgcn_exp2f(hi);
  // overflow, underflow, infinities and NaN: e alone is the answer (lo may be NaN there)
  return fabsf(hi) < 128.f ? fmaf(e, lo * kLn2, e) : e;
}

// The gate's a, and what multiplies u in b (1 for a log gate).
template <int KIND>
__device__ __forceinline__ void gate_terms(float g, float& a, float& c) {
  if constexpr (KIND == SSDQ_GATE_LOG) {
    a = exp_f32(g);
    c = 1.f;
  } else {
    // with e = exp(-|g|) both sigmoids keep their relative precision on either side
    const float e = exp_f32(-fabsf(g));
    const float small = 1.f + e;
    float inv = __builtin_amdgcn_rcpf(small);
    inv = fmaf(fmaf(-small, inv, 1.f), inv, inv);   // one Newton step: within an ulp
    const float low = e * inv;
    a = g < 0.f ? low : inv;
    c = g < 0.f ? inv : low;
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

// The code of v under scale s: the integer nearest to the exact quotient v / s, ties to even.
// k = rint(v rcp(s)) is one of the two nearest integers, since the product is within 2^-14 of the
// quotient, and v - k s is exact in one fma (|v - k s| stays near s / 2 and is a multiple of the
// smaller operand's last place), so comparing it with s / 2 decides the rest exactly.
struct CodeScale {
  float rcp, half, s;
};
__device__ __forceinline__ CodeScale code_scale(float s) {
  // a zero or NaN scale codes everything as 0
  const bool some = s > 0.f;
  return CodeScale{some ? __builtin_amdgcn_rcpf(s) : 0.f, some ? 0.5f * s : __builtin_inff(), some ? s : 0.f};
}
__device__ __forceinline__ int32_t code_of(float v, CodeScale c) {
  float k = rintf(v * c.rcp);
  const float r = fmaf(-k, c.s, v);
  if (fabsf(r) > c.half) k += r > 0.f ? 1.f : -1.f;
  // a tie between k and its neighbour: the even one
  else if (fabsf(r) == c.half && (int32_t(k) & 1)) k += r > 0.f ? 1.f : -1.f;
  return int32_t(k);
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
// The codes of V neighbouring elements under scale s, packed.
template <int V, typename P>
__device__ __forceinline__ typename Bytes<V>::type codes_of(const P& x, float s) {
  const CodeScale c = code_scale(s);
  struct { int8_t e[V]; } q;
#pragma unroll
  for (int v = 0; v < V; ++v) q.e[v] = int8_t(code_of(x[v], c));
  return __builtin_bit_cast(typename Bytes<V>::type, q);
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
