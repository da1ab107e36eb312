// Residual, RMS norm, rotation and int8 in one pass.
//
//   h = x + r;  y = h rsqrt(mean h^2 + eps) (w + offset);  int8 of the rotated y, a scale a token
//
// HBM bound: every value is read once and written once.  A workgroup holds a token in registers, 16
// consecutive values a lane as the rotation wants them (fwht256_row16), and passes two barriers: the
// sum of squares, then the largest rotated magnitude.  The next token's values are on their way
// meanwhile.  The sum is fp64 (products of fp32 numbers are exact in it), so the factor does not
// depend on how the sum is split, but for one rounding in some 2^28; it costs one conversion and one multiply-add a value.
#include <atomic>

#include "serve_internal.h"

namespace w4a8 {
namespace {

constexpr int kMaxThreads = 1024;
constexpr uint32_t kOutside = 0x80000000u;  // buffer offset past any row: reads zero, stores dropped
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 16 consecutive values as they lie in memory
template <bool BF16>
struct Raw16 {
    u32x4 a[BF16 ? 2 : 4];
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t element) {
        const uint32_t off = element == kOutside ? kOutside : element * (BF16 ? 2u : 4u);
#pragma unroll
        for (int i = 0; i < (BF16 ? 2 : 4); i++) a[i] = __builtin_amdgcn_raw_buffer_load_b128(r, off + 16u * i, 0, 0);
    }
    __device__ __forceinline__ void values(float v[16]) const {
#pragma unroll
        for (int i = 0; i < (BF16 ? 2 : 4); i++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if constexpr (BF16) {
                    v[8 * i + 2 * j] = __uint_as_float(a[i][j] << 16);
                    v[8 * i + 2 * j + 1] = __uint_as_float(a[i][j] & 0xFFFF0000u);
                } else {
                    v[4 * i + j] = __uint_as_float(a[i][j]);
                }
            }
    }
};

__device__ __forceinline__ void store16(__amdgpu_buffer_rsrc_t r, uint32_t element, bool bf16, const float v[16]) {
    if (bf16) {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const u32x4 o = {pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                             pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7])};
            __builtin_amdgcn_raw_buffer_store_b128(o, r, (element == kOutside ? kOutside : element * 2u) + 16u * i, 0, 0);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const u32x4 o = {__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])};
            __builtin_amdgcn_raw_buffer_store_b128(o, r, (element == kOutside ? kOutside : element * 4u) + 16u * i, 0, 0);
        }
    }
}

// Tokens blockIdx.x, blockIdx.x + gridDim.x, ...; R blocks of 256 a group of 16 lanes.
template <bool XB, bool RB, int R>
__global__ __launch_bounds__(kMaxThreads) void k_add_norm(NormArgs a) {
    __shared__ double s_sum[2][kMaxThreads / 64];
    __shared__ float s_top[2][kMaxThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
    const int groups = blockDim.x >> 4, t = tid & 15;
    const int nblk = (int)(a.K / kRot);
    uint32_t at[R];  // this lane's first element of each block; absent blocks are zeros and are not stored
#pragma unroll
    for (int r = 0; r < R; r++) {
        const int b = (tid >> 4) + r * groups;
        at[r] = b < nblk ? (uint32_t)(b * kRot + 16 * fwht_row16_nibble(t)) : kOutside;
    }
    auto row = [&](const void *base, int64_t m, int64_t stride, int64_t bytes) {  // a token past the last: empty
        const bool in = m < a.M;
        return __builtin_amdgcn_make_buffer_rsrc((void *)(static_cast<const char *>(base) + (in ? m : 0) * stride), (short)0,
                                                 in ? (int)bytes : 0, 0x00020000);
    };
    const bool has_r = a.r != nullptr;
    const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc((void *)a.w, (short)0, (int)(a.K * 4), 0x00020000);
    Raw16<false> w[R];
#pragma unroll
    for (int r = 0; r < R; r++) w[r].load(wr, at[r]);

    struct Token {
        Raw16<XB> x[R];
        Raw16<RB> r[R];
    };
    auto load = [&](int64_t m, Token &v) {
        const __amdgpu_buffer_rsrc_t rx = row(a.x, m, a.x_stride * (XB ? 2 : 4), a.K * (XB ? 2 : 4));
#pragma unroll
        for (int r = 0; r < R; r++) v.x[r].load(rx, at[r]);
        if (has_r) {
            const __amdgpu_buffer_rsrc_t rr = row(a.r, m, a.r_stride * (RB ? 2 : 4), a.K * (RB ? 2 : 4));
#pragma unroll
            for (int r = 0; r < R; r++) v.r[r].load(rr, at[r]);
        }
    };
    auto finish = [&](int64_t m, const Token &in, int par) {
        float v[R][16];
        double sum = 0.0;
#pragma unroll
        for (int r = 0; r < R; r++) {
            in.x[r].values(v[r]);
            if (has_r) {
                float y[16];
                in.r[r].values(y);
#pragma unroll
                for (int i = 0; i < 16; i++) v[r][i] = v[r][i] + y[i];
                if constexpr (RB) {
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const uint32_t p = pack_bf16(v[r][i], v[r][i + 1]);
                        v[r][i] = __uint_as_float(p << 16);
                        v[r][i + 1] = __uint_as_float(p & 0xFFFF0000u);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 16; i++) sum = fma((double)v[r][i], (double)v[r][i], sum);
        }
        if (a.h) {
            const __amdgpu_buffer_rsrc_t rh = row(a.h, m, a.K * (RB ? 2 : 4), a.K * (RB ? 2 : 4));
#pragma unroll
            for (int r = 0; r < R; r++) store16(rh, at[r], RB, v[r]);
        }
#pragma unroll
        for (int s = 32; s > 0; s >>= 1) sum += __shfl_xor(sum, s);
        if (lane == 0) s_sum[par][wave] = sum;
        __syncthreads();
        sum = s_sum[par][0];
        for (int i = 1; i < waves; i++) sum += s_sum[par][i];
        const float f = (float)(1.0 / sqrt(sum / (double)a.K + a.eps));
#pragma unroll
        for (int r = 0; r < R; r++) {
            float wv[16];
            w[r].values(wv);
#pragma unroll
            for (int i = 0; i < 16; i++) v[r][i] = v[r][i] * f * (wv[i] + a.offset);
        }
        if (a.normed) {
            const int64_t bytes = a.K * (a.normed_bf16 ? 2 : 4);
            const __amdgpu_buffer_rsrc_t rn = row(a.normed, m, bytes, bytes);
#pragma unroll
            for (int r = 0; r < R; r++) store16(rn, at[r], a.normed_bf16, v[r]);
        }
        if (!a.x_q) return;
        // as k_prepare_tokens has it
        float top = 0.0f;
#pragma unroll
        for (int r = 0; r < R; r++) {
            fwht256_row16(v[r], t);
#pragma unroll
            for (int i = 0; i < 16; i++) top = fmaxf(top, fabsf(v[r][i]));
        }
#pragma unroll
        for (int s = 32; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor(top, s));
        if (lane == 0) s_top[par][wave] = top;
        __syncthreads();
        top = s_top[par][0];
        for (int i = 1; i < waves; i++) top = fmaxf(top, s_top[par][i]);
        const float s = top / 127.0f, rs = s >= kQuantFastMin ? 1.0f / s : 0.0f;
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(s), row(a.s_x, m, 4, 4), tid == 0 ? 0u : kOutside, 0, 0);
        const __amdgpu_buffer_rsrc_t rq = row(a.x_q, m, a.K, a.K);
#pragma unroll
        for (int r = 0; r < R; r++) {
            const uint4 q = top > 0.0f ? quant16_auto(v[r], s, rs) : make_uint4(0, 0, 0, 0);
            __builtin_amdgcn_raw_buffer_store_b128(u32x4{q.x, q.y, q.z, q.w}, rq, at[r], 0, 0);
        }
    };

    // a thread reads s_sum[par] and s_top[par] before the next token's first barrier and they are written
    // again one token later, after it
    const int64_t step = gridDim.x;
    int64_t m = blockIdx.x;  // < M: the grid is at most M
    if constexpr (R == 1) {
        Token A, B;
        load(m, A);
        for (;;) {
            load(m + step, B);
            finish(m, A, 0);
            m += step;
            if (m >= a.M) break;
            load(m + step, A);
            finish(m, B, 1);
            m += step;
            if (m >= a.M) break;
        }
    } else {
        // longer rows: the registers hold one token
        for (int par = 0; m < a.M; m += step, par ^= 1) {
            Token A;
            load(m, A);
            finish(m, A, par);
        }
    }
}

template <bool XB, bool RB, int R>
hipError_t launch_r(const NormArgs &a, int num_cu, unsigned threads, hipStream_t stream) {
    // as many workgroups as the card holds at once (looked up once per size)
    static std::atomic<int> per_cu[kMaxThreads / 64 + 1];
    int pc = per_cu[threads / 64].load(std::memory_order_relaxed);
    if (pc == 0) {
        const hipError_t e = hipOccupancyMaxActiveBlocksPerMultiprocessor(&pc, k_add_norm<XB, RB, R>, (int)threads, 0);
        if (e != hipSuccess) return e;
        if (pc < 1) pc = 1;
        per_cu[threads / 64].store(pc, std::memory_order_relaxed);
    }
    const int64_t most = (int64_t)num_cu * pc;
    k_add_norm<XB, RB, R><<<(unsigned)(a.M < most ? a.M : most), threads, 0, stream>>>(a);
    return hipGetLastError();
}

template <bool XB, bool RB>
hipError_t launch_t(const NormArgs &a, int num_cu, hipStream_t stream) {
    const int64_t nblk = a.K / kRot, need = (nblk * 16 + kMaxThreads - 1) / kMaxThreads, rounds = need <= 2 ? need : 4;
    const unsigned threads = (unsigned)(((nblk + rounds - 1) / rounds * 16 + 63) / 64 * 64);
    switch (rounds) {
        case 1: return launch_r<XB, RB, 1>(a, num_cu, threads, stream);
        case 2: return launch_r<XB, RB, 2>(a, num_cu, threads, stream);
        default: return launch_r<XB, RB, 4>(a, num_cu, threads, stream);
    }
}

}  // namespace

hipError_t launch_add_norm(const NormArgs &a, int x_bf16, int r_bf16, int num_cu, hipStream_t stream) {
    if (x_bf16) return r_bf16 ? launch_t<true, true>(a, num_cu, stream) : launch_t<true, false>(a, num_cu, stream);
    return r_bf16 ? launch_t<false, true>(a, num_cu, stream) : launch_t<false, false>(a, num_cu, stream);
}

}  // namespace w4a8
