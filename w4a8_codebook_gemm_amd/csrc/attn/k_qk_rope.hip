// Head norm and rotary positions of queries and keys, one pass.
//
//   y = x * rsqrt(mean x^2 + eps) * (w + offset);  (a, b) -> (a c - b s, b c + a s)
//
// HBM bound: every value is read and written once, some 10 flops each.  A head is held by
// head_dim / 8 lanes, 8 consecutive values a lane (16 bytes of bf16, 32 of fp32), so the sum
// of squares is a few lane exchanges and a rotated pair is in one lane (interleaved) or in
// lanes R / 16 apart (half layout; R is a multiple of 16).  The angles do not depend on the
// head: a wave takes one token, computes its cosines and sines once, a lane or two lanes' worth
// of angles each, and keeps those of its eight values in registers for all heads it passes
// over.  The angle is position * inv_freq in turns, reduced to [-1/2, 1/2] in fp64 (at position
// 2^18 an fp32 product is off by 2^-7 of a radian); sine and cosine of its fp32 part are fp32, what that
// part leaves out is added to both.
//
// Measured: 8192 tokens, 24 + 4 heads of 256, fp32 to bf16, 77.5 us, 4.5 TB/s (a large copy runs at 4.75 here); 1021 tokens,
// 32 + 8 of 128, fp32, 13.6 us, 3.0 TB/s, of it 4.4 us that a call of one token takes as well.
#include "attn_internal.h"

namespace w4a8 {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 2;  // passes whose loads are in flight

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

// Streamed past the caches: measured 2 to 7% faster from 2048 tokens on, the same below.
template <bool BF16>
__device__ __forceinline__ void store8(void *y, int64_t off, const float v[8]) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    if constexpr (BF16) {
        const u32x4 w = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(y) + off));
    } else {
        u32x4 *p = reinterpret_cast<u32x4 *>(static_cast<float *>(y) + off);
        const u32x4 w = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
        const u32x4 z = {__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
        __builtin_nontemporal_store(w, p);
        __builtin_nontemporal_store(z, p + 1);
    }
}

// Wave w of the grid: token w / chunks, passes (w % chunks) * per .. + per - 1 of its passes over the query
// heads followed by those over the key heads; a pass is 64 / kLanes heads.
template <int D, bool XB, bool YB>
__global__ __launch_bounds__(kThreads) void k_qk_norm_rope(RopeArgs a, int chunks, int per) {
    constexpr int kLanes = D / 8;         // lanes of a head
    constexpr int kHeads = 64 / kLanes;   // heads a pass
    __shared__ float s_cs[kThreads / 64][2][D / 2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = a.rotary / 2;
    const int64_t gw = (int64_t)blockIdx.x * (kThreads / 64) + wave;
    const int64_t m = gw / chunks;
    if (m >= a.M) return;
    const int from = (int)(gw - m * chunks) * per;
    const int pq = (a.q.heads + kHeads - 1) / kHeads, pk = (a.k.heads + kHeads - 1) / kHeads;
    const int l = lane % kLanes, d = 8 * l, sub = lane / kLanes;

    // this lane's factors: y = u c + partner s, the sign in s; 1 and 0 behind the rotated part
    float c[8], s[8];
    {
        const double pos = (double)a.positions[m];
        float *cs = s_cs[wave][0], *sn = s_cs[wave][1];
        for (int i = lane; i < half; i += 64) {
            const double turns = pos * (a.inv_freq[i] * 0.15915494309189533577);
            // what the fp32 angle leaves out, in radians, is small enough for one term
            const double part = turns - rint(turns);
            const float near = (float)part, rest = (float)((part - (double)near) * 6.28318530717958647692);
            float sv, cv;
            sincospif(2.0f * near, &sv, &cv);
            cs[i] = fmaf(-rest, sv, cv) * a.attn_factor;
            sn[i] = fmaf(rest, cv, sv) * a.attn_factor;
        }
        // the wave reads what its own lanes wrote
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int k = a.interleaved ? 4 * l + (i >> 1) : (d < half ? d : d - half) + i;
            const bool first = a.interleaved ? (i & 1) == 0 : d < half;
            c[i] = d < a.rotary ? cs[k] : 1.0f;
            s[i] = d < a.rotary ? (first ? -sn[k] : sn[k]) : 0.0f;
        }
    }
    const int partner = d >= a.rotary ? lane : d < half ? lane + half / 8 : lane - half / 8;

    auto run = [&](const w4a8_heads &p, int pa, int pb) {  // passes pa .. pb - 1 over the heads of p
        if (pa >= pb) return;
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; i++) w[i] = p.weight ? p.weight[d + i] + a.offset : 1.0f;
        const int64_t x0 = m * p.token_stride + d, y0 = m * p.heads * D + d;
        // lanes past the last head read it and do not store
        auto load = [&](int i, float v[8]) {
            const int h = i * kHeads + sub;
            load8<XB>(p.x, x0 + (h < p.heads ? h : p.heads - 1) * p.head_stride, v);
        };
        float v[kAhead][8];
#pragma unroll
        for (int z = 0; z < kAhead; z++)
            if (pa + z < pb) load(pa + z, v[z]);
        for (int i0 = pa; i0 < pb; i0 += kAhead) {
#pragma unroll
            for (int z = 0; z < kAhead; z++) {
                const int i = i0 + z;
                if (i >= pb) break;
                float u[8], y[8];
#pragma unroll
                for (int j = 0; j < 8; j++) u[j] = v[z][j];
                if (i + kAhead < pb) load(i + kAhead, v[z]);
                if (p.weight) {
                    float ss = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; j++) ss = fmaf(u[j], u[j], ss);
#pragma unroll
                    for (int t = 1; t < kLanes; t <<= 1) ss += __shfl_xor(ss, t);
                    const float r = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
                    for (int j = 0; j < 8; j++) u[j] = u[j] * r * w[j];
                }
                if (a.interleaved) {
#pragma unroll
                    for (int j = 0; j < 8; j++) y[j] = fmaf(u[j ^ 1], s[j], u[j] * c[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; j++) y[j] = fmaf(__shfl(u[j], partner), s[j], u[j] * c[j]);
                }
                const int h = i * kHeads + sub;
                if (h < p.heads) store8<YB>(p.out, y0 + h * D, y);
            }
        }
    };
    const int to = from + per < pq + pk ? from + per : pq + pk;
    run(a.q, from, to < pq ? to : pq);
    run(a.k, from > pq ? from - pq : 0, to - pq);
}

template <int D>
hipError_t launch_d(const RopeArgs &a, int xb, int yb, int num_cu, hipStream_t stream) {
    constexpr int kHeads = 64 / (D / 8), kWaves = kThreads / 64;
    const int passes = (a.q.heads + kHeads - 1) / kHeads + (a.k.heads + kHeads - 1) / kHeads;
    // a wave for all of a token's passes where that gives each SIMD four waves, else as few as give
    // them that
    const int64_t want = 16 * (int64_t)num_cu;
    int chunks = (int)(a.M >= want ? 1 : (want + a.M - 1) / a.M);
    if (chunks > passes) chunks = passes;
    const int per = (passes + chunks - 1) / chunks;
    chunks = (passes + per - 1) / per;
    const unsigned grid = (unsigned)((a.M * chunks + kWaves - 1) / kWaves);
    auto f = xb ? (yb ? k_qk_norm_rope<D, true, true> : k_qk_norm_rope<D, true, false>)
                : (yb ? k_qk_norm_rope<D, false, true> : k_qk_norm_rope<D, false, false>);
    f<<<grid, kThreads, 0, stream>>>(a, chunks, per);
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
