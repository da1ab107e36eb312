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

// Probabilities of bf16 rows enter the second product as one fp16 number, 11 bits where the output has 8: over 777 positions
// that moves the output by 0.0002 of itself before its own rounding, and the error against 64 bits from 0.00166 to 0.00167; a
// second number would make a prompt's products half as many again.  fp32 rows have two.

// The running maximum m, a whole number, after a largest exponent t = s fac.  Exponents are one multiply-add each,
// s fac - m, which does not round the product as t is rounded: m is 2^-22 of t above it (2 to 4 of its last places),
// so that none of them passes 0 by rounding.  For |t| up to 2^16 that is 2^-6 before it is rounded up; from 2^26 on it takes a row's
// weights out of fp16's range.  Where m has to grow it grows by kAhead more, so that it seldom does: the weights
// and sums so far are rescaled each time, D / 2 multiplications a lane.  The largest weight then stands at 2^(kProbExp - 1 - kAhead)
// or more.  0 and 3 ahead: prompts 2 x 2048 of heads of 256 1449 and 1430 us, 8192 of 128 591 and 582, fp32 4096 of 64 93.5 and 91.5; single tokens
// alike.  (Where nothing is seen t is -inf, the number above it is none, and m stays.)
constexpr float kAhead = 3.0f;
__device__ __forceinline__ float running_maximum(float m, float t) {
    const float w = ceilf(fmaf(fabsf(t), 0x1p-22f, t));
    return w > m ? w + kAhead : m;
}

}  // namespace w4a8
