// Operand fragments of the matrix core made from a cache in 4 bits, exactly.
//
// A value is e2m1 * sc * unit: two significant bits times five.  The scale byte b, shifted to b << 6,
// is the fp16 number sc(b) 2^-18 whatever the byte is (its exponent field ends below fp16's infinities), and one
// instruction makes two codes e2m1 * 2^8 in fp16; the packed product, value / unit * 2^-10, lies between 2^-11
// and 2976 and is a normal fp16 number or zero.  The unit is the caller's.
#pragma once

#include "../attn/attn_tiles.h"
#include "serve_internal.h"

namespace w4a8 {

constexpr int kValueExp = 10;  // fragments are value / unit * 2^-kValueExp

// Two codes (byte J) as fp16, times s.
template <int J>
__device__ __forceinline__ uint32_t codes_times(uint32_t w, half2_t s) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.0f, J)) * s);
}

// Byte J of a dword of scale bytes for two values that share it, and bytes J and J + 1 for one each.
template <int J>
__device__ __forceinline__ half2_t scale_both(uint32_t w) {
    return __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0u, w, 0x0C000C00u | (uint32_t)J | (uint32_t)J << 16) << 6);
}
template <int J>
__device__ __forceinline__ half2_t scale_pair(uint32_t w) {
    return __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0u, w, 0x0C000C00u | (uint32_t)J | (uint32_t)(J + 1) << 16) << 6);
}

// Eight consecutive values of one token.
__device__ __forceinline__ half8_t values_natural(uint32_t w, half2_t s) {
    return __builtin_bit_cast(half8_t, make_uint4(codes_times<0>(w, s), codes_times<1>(w, s), codes_times<2>(w, s), codes_times<3>(w, s)));
}

// The codes of two tokens' dwords side by side: a byte holds both tokens' code of one value, the first
// token's low; even values 0, 2, 4, 6 and odd values 1, 3, 5, 7.
__device__ __forceinline__ uint32_t even_codes(uint32_t first, uint32_t second) { return (first & 0x0F0F0F0Fu) | ((second << 4) & 0xF0F0F0F0u); }
__device__ __forceinline__ uint32_t odd_codes(uint32_t first, uint32_t second) { return ((first >> 4) & 0x0F0F0F0Fu) | (second & 0xF0F0F0F0u); }

// Whether a row's exponents s fac - m may not be one multiply-add: it does not round the product, which then
// may pass a maximum m that was rounded by 2^-24 of itself.  Up to this size that is 2^-8, above it the product is rounded first.
__device__ __forceinline__ bool far_scores(float m) { return fabsf(m) > 65536.0f && m > kLow; }

}  // namespace w4a8
