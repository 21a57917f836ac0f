// Layout and number format of the paged 8-bit key / value cache.
//
// A page holds 64 tokens of one head: 64·dim E4M3 codes of K, as many of V, and one exponent
// byte each (value = code · 2^(byte − 127)).  The codes are stored in the order in which the
// attention kernel's matrix instructions take them, in fragments of 1 KB: 16 bytes for each of
// the 64 lanes, so that a page is read with whole, contiguous requests and its LDS image needs
// no swizzle (lane l reads bytes 16 l on: every bank once).
//
//   K, code (token t, channel d): fragment ((t/32)·(dim/64) + d/64)·2 + (d/16)%2,
//      lane 32·((d/32)%2) + t%32, byte d%16 — eight bytes are, widened, a lane's operand of a
//      32x32x16 bf16 MFMA, whose channels are then 8 of each half of a block of 64.
//   V, code (token t, channel d): fragment (d/32)·2 + t/32, lane 32·((t/4)%2) + d%32,
//      byte 8·((t/16)%2) + 4·((t/8)%2) + t%4 — two operands of a 32x32x16 bf16 MFMA whose eight
//      tokens per lane are those that the product K·Qᵀ leaves in one lane's registers.
#pragma once

#include "device.h"

namespace svdq {

constexpr int kPage = 64;                    // tokens
constexpr int kExpMin = -110, kExpMax = 119; // exponents of a page's scale

__device__ __forceinline__ int k_offset(int t, int d, int dim) {
  const int frag = ((t >> 5) * (dim >> 6) + (d >> 6)) * 2 + ((d >> 4) & 1);
  return (frag * 64 + ((d >> 5) & 1) * 32 + (t & 31)) * 16 + (d & 15);
}

__device__ __forceinline__ int v_offset(int t, int d) {
  const int frag = (d >> 5) * 2 + (t >> 5);
  return (frag * 64 + ((t >> 2) & 1) * 32 + (d & 31)) * 16 + ((t >> 4) & 1) * 8 +
         ((t >> 3) & 1) * 4 + (t & 3);
}

constexpr uint32_t kInfBits = 0x7F80;        // |bf16| from here on: infinity or NaN

// The larger of two bf16 magnitudes (sign bits clear) in each half.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a),
                                                                __builtin_bit_cast(u16x2_t, b)));
}

// Smallest e with a <= 448·2^e, within [kExpMin, kExpMax] (448 = 0.875·2^9).
__device__ __forceinline__ int page_exponent(float a) {
  if (!(a > 0.0f)) return kExpMin;
  const float m = __builtin_amdgcn_frexp_mantf(a);
  const int x = __builtin_amdgcn_frexp_expf(a);
  const int e = m <= 0.875f ? x - 9 : x - 8;
  return e < kExpMin ? kExpMin : (e > kExpMax ? kExpMax : e);
}

// 2^e for -126 <= e <= 127
__device__ __forceinline__ float two_to(int e) {
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

}  // namespace svdq
