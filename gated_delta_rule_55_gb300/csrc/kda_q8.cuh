// Rows of a cache kept in 8 bits: D numbers of e4m3 and one byte e for a token's key or value of a
// kv head, which stand for number * 2^(e - 127).
//
// The scale is a power of two: e4m3 numbers have steps relative to their size, so a scale in
// between would keep no more of them, while powers of two make the scaling, and all that reads the
// row back (a bf16 holds number * scale exactly), free of rounding.  Of the powers, the smallest
// whose 448-fold (the largest e4m3) reaches the row's largest magnitude: numbers lose steps only
// where they are less than 2^-14 of it.
#pragma once

#include <cuda_fp16.h>

#include "kda_internal.cuh"

namespace kda {
namespace q8 {

constexpr int kBias = 127;
// Exponents of a scale: 448 * 2^119 is the largest fp32, and the smallest number 2^-9 * 2^-110
// is still a normal bf16 (rows below that keep what of them is above it).
constexpr int kLo = -110, kHi = 119;
constexpr int kNaN = 255;  // the byte of a row that held an infinity or a NaN: all of it is NaN

// The scale's exponent for a row whose largest magnitude has these bits (finite).
__device__ __forceinline__ int exponent(uint32_t top) {
  // top = m 2^x, 1 <= m < 2: x - 8, or one more where m > 1.75 (448 = 1.75 * 2^8)
  const int e = (int)((top + 0x1fffffu) >> 23) - 127 - 8;
  return min(max(e, kLo), kHi);
}
__device__ __forceinline__ float power(int e) {  // 2^e, -126 <= e <= 127
  return __uint_as_float((uint32_t)(e + 127) << 23);
}
// Two numbers as e4m3, to nearest (halves to even), the first in the lower byte.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint32_t x) {  // its lower two bytes
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)x));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// What a byte multiplies its numbers by, in fp32 (exact; 0 stands for 2^-127).
__device__ __forceinline__ float scale(uint32_t byte) {
  return byte == kNaN ? __uint_as_float(0x7fc00000u)
                      : __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
}

// The same for 16 numbers in bf16, for the tensor cores.  A number's bits, spread over a bf16's
// (sign; four exponent bits, the lower ones; three mantissa bits, the upper ones), are those of
// the number times 2^-120, e4m3's subnormals becoming bf16's, so that one product with
// 2^(120 + e - 127) makes it what it stands for.  Where that is no bf16 (e > 7 + 127) a second one
// follows.
struct Scale16 {
  uint32_t m;     // 2^(byte - 7) twice (or 2^127, or NaN)
  uint32_t more;  // 2^(byte - 134), where m is 2^127
  bool big;
  __device__ __forceinline__ explicit Scale16(uint32_t byte) {
    big = byte > 134 && byte != kNaN;
    const uint32_t x = byte == kNaN ? 0x7fc0u : min(byte + 120u, 254u) << 7;
    const uint32_t y = big ? (byte - 7u) << 7 : 0x3f80u;
    m = x | x << 16;
    more = y | y << 16;
  }
};
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Four numbers (a register of them) as two registers of bf16 pairs: the first and third, the second
// and fourth (place()).  In this order a number's bits move by the same distance in both halves of a
// register, and half of the moves are products by powers of two, which pass beside the logic
// operations.  (The first product: a caller that may meet big scales makes the second.)
__device__ __forceinline__ void expand4(uint32_t w, const Scale16& s, uint32_t& even,
                                        uint32_t& odd) {
  constexpr uint32_t kSign = 0x80008000u, kRest = 0x07f007f0u;
  even = mul_bf16x2((w * 256u & kSign) | (w * 16u & kRest), s.m);
  odd = mul_bf16x2((w & kSign) | (w >> 4 & kRest), s.m);
}
__device__ __forceinline__ constexpr int place(int i) {  // of number i among the results
  return (i & ~3) | (i & 1) << 1 | (i >> 1 & 1);
}

__device__ __forceinline__ void expand4_in_order(uint32_t w, const Scale16& s, uint32_t& lo,
                                                 uint32_t& hi) {
  const uint32_t x = __byte_perm(w, 0, 0x1404), y = __byte_perm(w, 0, 0x3424);  // b << 8
  lo = mul_bf16x2((x & 0x80008000u) | (x >> 4 & 0x07f007f0u), s.m);
  hi = mul_bf16x2((y & 0x80008000u) | (y >> 4 & 0x07f007f0u), s.m);
}

}  // namespace q8
}  // namespace kda
