// Warp-level matrix products of 16-bit operands into fp32, and the exact splits that
// carry fp32 operands through them (few_tokens.cu, adapters.cu).
#pragma once

#include <math.h>

#include "rows.cuh"

namespace moe {

// d += a (16 x 16, rows g and g + 8 of a lane, g = lane / 4) * b (16 x 8, column g)
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], uint32_t a0, uint32_t a1,
                                                        uint32_t a2, uint32_t a3, uint32_t b0,
                                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], uint32_t a0, uint32_t a1,
                                                 uint32_t a2, uint32_t a3, uint32_t b0,
                                                 uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The power of two that brings a value of magnitude m into [2^13, 2^14), as its fp32
// bits: room for fp16 operands whose products with a 16-bit number are added up.  1
// where m is zero, infinite or NaN; inside 2^-126 .. 2^126, so that its inverse,
// 1 / 2^e, is a normal number too.
__device__ __forceinline__ uint32_t fp16_range_bits(uint32_t m_bits) {
  const int e = (int)(m_bits >> 23) & 0xff;
  if ((m_bits & 0x7fffffffu) == 0u || e == 255) return 127u << 23;
  return (uint32_t)min(267 - e, 253) << 23;
}
__device__ __forceinline__ float inverse_pow2(uint32_t bits) {
  return __uint_as_float((254u << 23) - bits);
}

// The fp32 bits of |v| as they count towards a largest magnitude: what is not finite does not.
__device__ __forceinline__ uint32_t magnitude(float v) {
  const uint32_t bits = __float_as_uint(fabsf(v));
  return bits < 0x7f800000u ? bits : 0u;
}

// What a 16-bit term leaves of v: nothing of an infinity, which would be NaN, nor of a NaN.
__device__ __forceinline__ float left_of(float v, float term) {
  return fabsf(term) < INFINITY ? v - term : 0.f;
}

// (lo, hi) rounded to the 16-bit type, and what that rounding left, rounded again.
template <typename T>
__device__ __forceinline__ void split2(float lo, float hi, uint32_t& first, uint32_t& rest) {
  first = pack2<T>(lo, hi);
  const float2 f = unpack2<T>(first);
  rest = pack2<T>(left_of(lo, f.x), left_of(hi, f.y));
}

}  // namespace moe
