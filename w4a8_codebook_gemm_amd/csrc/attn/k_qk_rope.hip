// Head norm and rotary positions of queries and keys, one pass.
//
//   y = x * rsqrt(mean x^2 + eps) * (w + offset);  (a, b) -> (a c - b s, b c + a s)
//
// HBM bound: every value is read and written once, some 10 flops each.  A head is held by
// head_dim / 8 lanes, 8 consecutive values a lane (16 bytes of bf16, 32 of fp32), so the sum
// of squares is a few lane exchanges and a rotated pair is in one lane (interleaved) or in
// lanes R / 16 apart (half layout; R is a multiple of 16).  The angles do not depend on the
// head: a workgroup takes whole tokens, computes R / 2 cos / sin a token into LDS once
// and reads them for all of the token's heads.  The angle is position * inv_freq in turns,
// reduced to [-1/2, 1/2] in fp64 (at position 2^18 an fp32 product is off by 2^-7 of a radian),
// its sine and cosine in fp32.
#include "attn_internal.h"

namespace w4a8 {
namespace {

constexpr int kThreads = 256;

template <bool BF16>
__device__ __forceinline__ void load8(const void *x, int64_t off, float v[8]) {
    if constexpr (BF16) {
        const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + off);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(x) + off);
        const float4 a = p[0], b = p[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}

template <bool BF16>
__device__ __forceinline__ void store8(void *y, int64_t off, const float v[8]) {
    if constexpr (BF16) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++)
            w[i] = (uint32_t)f32_to_bf16_rne(v[2 * i]) | (uint32_t)f32_to_bf16_rne(v[2 * i + 1]) << 16;
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(y) + off) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(y) + off);
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

// Workgroup (x, y): tokens x * T .. x * T + T - 1, heads y * chunk .. y * chunk + chunk - 1 of
// the query heads followed by the key heads.
template <int D, bool XB, bool YB>
__global__ __launch_bounds__(kThreads) void k_qk_norm_rope(RopeArgs a, int T, int chunk) {
    constexpr int kLanes = D / 8;            // lanes of a head
    constexpr int kHeads = kThreads / kLanes;  // heads a pass
    __shared__ float s_cos[4 * D / 2], s_sin[4 * D / 2];  // [T <= 4][R / 2]
    const int tid = threadIdx.x, half = a.rotary / 2;
    const int64_t m0 = (int64_t)blockIdx.x * T;
    const int nt = a.M - m0 < T ? (int)(a.M - m0) : T;
    for (int i = tid; i < nt * half; i += kThreads) {
        const double turns = (double)a.positions[m0 + i / half] * (a.inv_freq[i % half] * 0.15915494309189533577);
        float sn, cs;
        sincospif(2.0f * (float)(turns - rint(turns)), &sn, &cs);
        s_cos[i] = cs * a.attn_factor;
        s_sin[i] = sn * a.attn_factor;
    }
    const int heads = a.q.heads + a.k.heads;
    const int h0 = blockIdx.y * chunk;
    const int nh = heads - h0 < chunk ? heads - h0 : chunk;
    const int l = tid % kLanes, d = 8 * l;
    float wq[8], wk[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        wq[i] = a.q.weight ? a.q.weight[d + i] + a.offset : 1.0f;
        wk[i] = a.k.weight ? a.k.weight[d + i] + a.offset : 1.0f;
    }
    __syncthreads();
    // every lane of a wave runs every pass (lane exchanges below); lanes past the last head
    // work on the last one and do not store
    const int total = nt * nh;
    for (int base = 0; base < total; base += kHeads) {
        const int at = base + tid / kLanes;
        const int it = at < total ? at : total - 1;
        const int t = it / nh, h = h0 + it % nh;
        const bool isq = h < a.q.heads;
        const w4a8_heads &p = isq ? a.q : a.k;
        const int ph = isq ? h : h - a.q.heads;
        float v[8];
        load8<XB>(p.x, (m0 + t) * p.token_stride + ph * p.head_stride + d, v);
        if (p.weight) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; i++) ss = fmaf(v[i], v[i], ss);
#pragma unroll
            for (int s = 1; s < kLanes; s <<= 1) ss += __shfl_xor(ss, s);
            const float r = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = v[i] * r * (isq ? wq[i] : wk[i]);
        }
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] = v[i];
        if (a.interleaved) {
            if (d < a.rotary) {
                const float *cs = s_cos + t * half + 4 * l, *sn = s_sin + t * half + 4 * l;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    y[2 * i] = v[2 * i] * cs[i] - v[2 * i + 1] * sn[i];
                    y[2 * i + 1] = v[2 * i + 1] * cs[i] + v[2 * i] * sn[i];
                }
            }
        } else {
            const bool low = d < half;
            const int lane = tid & 63;
            const int partner = d < a.rotary ? (low ? lane + half / 8 : lane - half / 8) : lane;
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; i++) o[i] = __shfl(v[i], partner);
            if (d < a.rotary) {
                const float *cs = s_cos + t * half + (low ? d : d - half), *sn = s_sin + t * half + (low ? d : d - half);
#pragma unroll
                for (int i = 0; i < 8; i++) y[i] = low ? v[i] * cs[i] - o[i] * sn[i] : v[i] * cs[i] + o[i] * sn[i];
            }
        }
        if (at < total) store8<YB>(p.out, ((m0 + t) * p.heads + ph) * D + d, y);
    }
}

template <int D>
hipError_t launch_d(const RopeArgs &a, int xb, int yb, int num_cu, hipStream_t stream) {
    const int heads = a.q.heads + a.k.heads;
    constexpr int kHeads = kThreads / (D / 8);
    // few tokens: one pass a workgroup, heads spread over workgroups
    int T = 1, chunk = heads;
    if (a.M * ((heads + kHeads - 1) / kHeads) <= 4 * (int64_t)num_cu)
        chunk = kHeads;
    else if (a.M >= 4 * (int64_t)num_cu)
        T = 4;
    const dim3 grid((unsigned)((a.M + T - 1) / T), (unsigned)((heads + chunk - 1) / chunk));
    auto f = xb ? (yb ? k_qk_norm_rope<D, true, true> : k_qk_norm_rope<D, true, false>)
                : (yb ? k_qk_norm_rope<D, false, true> : k_qk_norm_rope<D, false, false>);
    f<<<grid, kThreads, 0, stream>>>(a, T, chunk);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_qk_norm_rope(const RopeArgs &a, int head_dim, int x_bf16, int out_bf16, int num_cu, hipStream_t stream) {
    switch (head_dim) {
        case 64: return launch_d<64>(a, x_bf16, out_bf16, num_cu, stream);
        case 128: return launch_d<128>(a, x_bf16, out_bf16, num_cu, stream);
        default: return launch_d<256>(a, x_bf16, out_bf16, num_cu, stream);
    }
}

}  // namespace w4a8
