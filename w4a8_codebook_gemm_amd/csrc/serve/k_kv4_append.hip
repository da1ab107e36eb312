// Append of keys and values into the paged cache in 4 bits.
//
// A group of 16 values is a lane's: its largest magnitude, its scale byte and its codes need no
// other lane.  A wave has 4 neighbouring groups of 16 tokens: rows are read in pieces of 128 bytes or
// more, and a group's scale bytes of tokens that follow each other, which lie together for values, are
// one store's.  The quotients are correctly rounded ones from the scale's reciprocal
// (quant4_r has the proof); two of them become codes in one instruction.
//
// HBM bound for large calls: 8192 tokens of 4 heads of 256, bf16, 10.2 us, 4.2 TB/s (its inputs past the caches 9.5), fp32
// 13.2; 65536 of 8 heads of 128 67.8, 5.1 TB/s; 61 tokens 2.9 us, which is a launch.  A copy runs at 5.39 TB/s here.
#include "serve_internal.h"

namespace w4a8 {
namespace {

constexpr int kThreads = 256;

// The nearest byte to t >= 0 by sc(byte), ties to even: 16 .. 32 steps of a power of two, or steps of 1.
__device__ __forceinline__ uint32_t scale_byte(float t) {
    t = fminf(t, 1e9f);
    int up = (int)(__float_as_uint(t) >> 23) - 131;  // t in [2^(up + 4), 2^(up + 5))
    up = up < 0 ? 0 : up > 14 ? 14 : up;
    const int b = 16 * up + (int)rintf(ldexpf(t, -up));
    return (uint32_t)(b < 1 ? 1 : b > 255 ? 255 : b);
}
__device__ __forceinline__ float scale_value(uint32_t b) {
    return b < 16 ? (float)b : ldexpf((float)(16 + (b & 15)), (int)(b >> 4) - 1);
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void k_kv4_append(Append4Args a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int D = a.c.head_dim, quads = D / 64, P = a.c.page_size;
    const int per = 2 * a.c.kv_heads * quads;  // waves of 16 tokens
    const int64_t w = (int64_t)blockIdx.x * (kThreads / 64) + wave;
    const int64_t tile = w / per;
    int rest = (int)(w - tile * per);
    const int64_t token = tile * 16 + (lane >> 2);
    if (token >= a.M) return;
    const int quad = rest % quads;
    rest /= quads;
    const int h = rest % a.c.kv_heads, kind = rest / a.c.kv_heads;
    const int grp = 4 * quad + (lane & 3);

    const int64_t slot = a.slots[token];
    float x[16];
    load16<BF16>(a.x[kind], token * a.stride[kind] + (int64_t)h * D + 16 * grp, x);
    const float unit = (kind ? a.c.v_unit : a.c.k_unit)[h];
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i++) top = fmaxf(top, fabsf(x[i]));
    const uint32_t b = scale_byte(top / (6.0f * unit));
    const float s = scale_value(b) * unit;
    float y[16];
    if (s >= kQuantFastMin && s <= 0x1p100f && top <= 8.0f * s) {
        const float r = 1.0f / s;
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const float q = x[i] * r;
            y[i] = copysignf(fmaf(fmaf(-q, s, x[i]), r, q), x[i]);  // (the sum of two zeros loses the sign)
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; i++) y[i] = x[i] / s;
    }
    uint32_t lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, y[0], y[1], 1.0f, 0);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, y[2], y[3], 1.0f, 1);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, y[4], y[5], 1.0f, 2);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, y[6], y[7], 1.0f, 3);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi, y[8], y[9], 1.0f, 0);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi, y[10], y[11], 1.0f, 1);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi, y[12], y[13], 1.0f, 2);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi, y[14], y[15], 1.0f, 3);
    if (slot < 0 || slot >> a.page_shift >= a.c.num_pages) return;
    const int64_t blk = (slot >> a.page_shift) * a.c.kv_heads + h;
    const int place = (int)(slot & (P - 1));
    *reinterpret_cast<uint2 *>((kind ? a.c.v : a.c.k) + (blk * P + place) * (D / 2) + 8 * grp) = make_uint2(lo, hi);
    if (kind) a.c.v_scale[(blk * (D / 16) + grp) * P + place] = (uint8_t)b;
    else a.c.k_scale[(blk * P + place) * (D / 16) + grp] = (uint8_t)b;
}

}  // namespace

hipError_t launch_kv4_append(const Append4Args &a, int bf16, hipStream_t stream) {
    constexpr int kWaves = kThreads / 64;
    const int64_t waves = (a.M + 15) / 16 * (2 * a.c.kv_heads * (a.c.head_dim / 64));
    const int64_t grid = (waves + kWaves - 1) / kWaves;
    if (bf16) k_kv4_append<true><<<(unsigned)grid, kThreads, 0, stream>>>(a);
    else k_kv4_append<false><<<(unsigned)grid, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace w4a8
