// Layout and number format of the paged 4-bit key / value cache.
//
// A page holds 64 tokens of one head.  A token's channels are quantised in blocks of 32 by the MXFP4
// rule (E2M1 codes under one power of two, value = code·2^(byte − 127)), each token by itself: an
// appended token changes no byte of another one, so nothing is rounded twice and tokens may be written
// in any order.  Per page and head: 32·dim bytes of codes and 2·dim of scales, of K and of V each.
//
// The codes are stored in the order in which the attention kernel's matrix instructions take them, in
// fragments of 1 KB, 16 bytes for each of the 64 lanes.  A byte holds the channels (d, d + 1), d even
// in the low nibble.
//
//   K, (token t, channel d): fragment (t/32)·(dim/64) + d/64, lane 32·((d/32)%2) + t%32, byte (d%32)/2:
//      a lane has one scale's block of one token, four operands of a 32x32x16 bf16 MFMA whose channels
//      are then 8 of each half of a block of 64.
//      Scale: byte lane·(dim/32) + fragment, so that a lane's scales of a page are one word.
//   V, (token t, channel d): fragment (d/64)·2 + t/32, lane 32·((t/4)%2) + (d/2)%32,
//      byte 8·((t/16)%2) + 4·((t/8)%2) + t%4: eight bytes are the eight tokens which the product K·Qᵀ
//      leaves in one lane's registers, at two channels; with the two channels apart they make operands
//      of two MFMAs.
//      Scale: byte ((d/32)·2 + (t/4)%2)·32 + 8·(t/16) + 4·((t/8)%2) + t%4, the order of the lane's
//      tokens.
#pragma once

#include "device.h"
#include "kv_layout.h"

namespace svdq {

// Exponents of a block's scale.  Six times the largest is summed over 2^31 tokens with weights of up
// to 2^8 without leaving fp32; the least is far above the numbers that fp32 cannot scale exactly.
constexpr int kExp4Min = -110, kExp4Max = 85;
constexpr uint32_t kNan4 = 255;  // scale byte of a block that holds an infinity or NaN

__device__ __forceinline__ int k4_offset(int t, int d, int dim) {
  const int frag = (t >> 5) * (dim >> 6) + (d >> 6), lane = ((d >> 5) & 1) * 32 + (t & 31);
  return (frag * 64 + lane) * 16 + ((d & 31) >> 1);
}
__device__ __forceinline__ int k4_scale_offset(int t, int d, int dim) {
  const int frag = (t >> 5) * (dim >> 6) + (d >> 6), lane = ((d >> 5) & 1) * 32 + (t & 31);
  return lane * (dim >> 5) + frag;
}
__device__ __forceinline__ int v4_offset(int t, int d) {
  const int frag = (d >> 6) * 2 + (t >> 5), lane = ((t >> 2) & 1) * 32 + ((d >> 1) & 31);
  return (frag * 64 + lane) * 16 + ((t >> 4) & 1) * 8 + ((t >> 3) & 1) * 4 + (t & 3);
}
__device__ __forceinline__ int v4_scale_offset(int t, int d) {
  return ((d >> 5) * 2 + ((t >> 2) & 1)) * 32 + (t >> 4) * 8 + ((t >> 3) & 1) * 4 + (t & 3);
}

// The scale operand of a conversion from byte `k` of a dword of scales.  The conversions read the
// exponent field alone: the bits that the shift leaves around it have no part (checked against
// every code), and the exponent 255 makes every code a NaN.
__device__ __forceinline__ float scale4(uint32_t w, int k) {
  return __uint_as_float(k == 3 ? w >> 1 : w << (23 - 8 * k));
}

// Two codes (byte `k` of a dword) times the scale, exactly, as a pair of bf16.
__device__ __forceinline__ uint32_t widen2(uint32_t w, int k, float scale) {
  return __builtin_bit_cast(uint32_t,
                            k == 0   ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)
                            : k == 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)
                            : k == 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)
                                     : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
}

// Two bf16 values divided by the scale as E2M1 codes (nearest even, at most ±6) in byte `k` of `old`.
__device__ __forceinline__ uint32_t code2(uint32_t old, uint32_t x, int k, float scale) {
  const bf16x2_t v = __builtin_bit_cast(bf16x2_t, x);
  return k == 0   ? __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, v, scale, 0)
         : k == 1 ? __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, v, scale, 1)
         : k == 2 ? __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, v, scale, 2)
                  : __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, v, scale, 3);
}

}  // namespace svdq
