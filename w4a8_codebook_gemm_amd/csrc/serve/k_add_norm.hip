// Residual, RMS norm, rotation and int8 in one pass.
//
//   h = x + r;  y = h rsqrt(mean h^2 + eps) (w + offset);  int8 of the rotated y, a scale a token
//
// HBM bound: every value is read once and written once.  A token is held in registers, 16 consecutive
// values a lane and block of 256 as the rotation wants them (fwht256_row16), by W waves of R blocks a
// group of 16 lanes.  Two numbers need all of a token: the sum of squares, then the largest rotated magnitude.
// One wave a token exchanges them between lanes alone, so nothing waits for another wave; more waves a token
// (fewer blocks a lane group) also meet at two barriers, and finish a single token sooner.
//
// The sum is fp64 (products of fp32 numbers are exact in it), so the factor does not depend on how the sum is
// split, but for one rounding in some 2^28.  Its root is the hardware's reciprocal square root and two Newton steps,
// y + y/2 (1 - a y^2), in fp64, as exact as a division by a root.  Largest relative error over 2^30 numbers of [1, 4), at four
// scales: 2^-24.2, 2^-47.7 after one step (which rounds the factor wrongly in one row of some 2^25), 2^-52.7 after two.
#include "serve_internal.h"

namespace w4a8 {
namespace {

constexpr int kMaxThreads = 1024;
constexpr uint32_t kOutside = 0x80000000u;  // buffer offset past any row: reads zero, stores dropped
constexpr int kMaxWeights = 32768;          // bytes of weights that a workgroup keeps in LDS
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

// Sum and maximum (of values >= 0) over a wave's lanes, by shifts within rows of 16, then from row to row; the last
// lane's, as uniform values.
template <int kCtrl, int kRows>
__device__ __forceinline__ uint32_t moved(uint32_t x) { return __builtin_amdgcn_update_dpp(0, (int)x, kCtrl, kRows, 0xF, false); }
template <int kCtrl, int kRows>
__device__ __forceinline__ double moved(double x) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    return __builtin_bit_cast(double, (uint64_t)moved<kCtrl, kRows>((uint32_t)b) | (uint64_t)moved<kCtrl, kRows>((uint32_t)(b >> 32)) << 32);
}
__device__ __forceinline__ double wave_sum(double x) {
    x += moved<0x111, 0xF>(x);  // row_shr:1, 2, 4, 8
    x += moved<0x112, 0xF>(x);
    x += moved<0x114, 0xF>(x);
    x += moved<0x118, 0xF>(x);
    x += moved<0x142, 0xA>(x);  // row_bcast:15, 31
    x += moved<0x143, 0xC>(x);
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)b, 63) |
                                          (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), 63) << 32);
}
template <int kCtrl, int kRows>
__device__ __forceinline__ float max_moved(float x) { return fmaxf(x, __uint_as_float(moved<kCtrl, kRows>(__float_as_uint(x)))); }
__device__ __forceinline__ float wave_max(float x) {
    x = max_moved<0x111, 0xF>(x);
    x = max_moved<0x112, 0xF>(x);
    x = max_moved<0x114, 0xF>(x);
    x = max_moved<0x118, 0xF>(x);
    x = max_moved<0x142, 0xA>(x);
    x = max_moved<0x143, 0xC>(x);
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(x), 63));
}

// 1 / sqrt(a), a > 0, normal and finite
__device__ __forceinline__ double reciprocal_root(double a) {
    double y = __builtin_amdgcn_rsq(a);
    y = fma(0.5 * y, fma(-a * y, y, 1.0), y);
    return fma(0.5 * y, fma(-a * y, y, 1.0), y);
}

// A workgroup has blockDim / 64 / W tokens at a time.  LW: the weights lie in LDS, as the lanes read them.  kThreads: most
// threads of a workgroup, for the registers.
template <bool XB, bool RB, int R, int kThreads, bool LW>
__global__ __launch_bounds__(kThreads, kThreads == 256 ? 4 : 1) void k_add_norm(NormArgs a, int W) {
    __shared__ double s_sum[2][kMaxThreads / 64];
    __shared__ float s_top[2][kMaxThreads / 64];
    __shared__ __attribute__((aligned(16))) char s_w[LW ? kMaxWeights : 16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int part = wave % W, tokens = waves / W;  // this wave's of its token's; tokens of the workgroup
    const int nblk = (int)(a.K / kRot);
    uint32_t at[R];  // this lane's first element of each block; absent blocks are zeros and are not stored
#pragma unroll
    for (int r = 0; r < R; r++) {
        const int b = r * 4 * W + 4 * part + (lane >> 4);
        at[r] = b < nblk ? (uint32_t)(b * kRot + 16 * fwht_row16_nibble(lane & 15)) : kOutside;
    }
    auto row = [&](const void *base, int64_t m, int64_t stride, int64_t bytes) {  // a token past the last: empty
        const bool in = m < a.M;
        return __builtin_amdgcn_make_buffer_rsrc((void *)(static_cast<const char *>(base) + (in ? m : 0) * stride), (short)0,
                                                 in ? (int)bytes : 0, 0x00020000);
    };
    const bool has_r = a.r != nullptr;
    const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc((void *)a.w, (short)0, (int)(a.K * 4), 0x00020000);
    // 16 bytes a lane, lanes side by side
    auto w_place = [&](int r, int i) { return reinterpret_cast<u32x4 *>(s_w) + (((r * W + part) * 4 + i) * 64 + lane); };
    if constexpr (LW) {
        if (wave < W) {
#pragma unroll
            for (int r = 0; r < R; r++) {
                Raw16<false> w;
                w.load(wr, at[r]);
#pragma unroll
                for (int i = 0; i < 4; i++) *w_place(r, i) = w.a[i];
            }
        }
        __syncthreads();
    }
    int par = 0;
    // a wave that is left over where W does not divide the waves, or stands behind the last token, goes along with empty rows
    for (int64_t m0 = (int64_t)blockIdx.x * tokens; m0 < a.M; m0 += (int64_t)gridDim.x * tokens, par ^= 1) {
        const int64_t m = wave / W < tokens ? m0 + wave / W : a.M;
        Raw16<XB> x[R];
        Raw16<RB> res[R];
        const __amdgpu_buffer_rsrc_t rx = row(a.x, m, a.x_stride * (XB ? 2 : 4), a.K * (XB ? 2 : 4));
#pragma unroll
        for (int r = 0; r < R; r++) x[r].load(rx, at[r]);
        if (has_r) {
            const __amdgpu_buffer_rsrc_t rr = row(a.r, m, a.r_stride * (RB ? 2 : 4), a.K * (RB ? 2 : 4));
#pragma unroll
            for (int r = 0; r < R; r++) res[r].load(rr, at[r]);
        }
        float v[R][16];
        double sum = 0.0;
#pragma unroll
        for (int r = 0; r < R; r++) {
            x[r].values(v[r]);
            if (has_r) {
                float y[16];
                res[r].values(y);
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
        // a wave reads s_sum[par] and s_top[par] before the next token's first barrier, and they are written
        // again one token later, behind it
        sum = wave_sum(sum);
        if (W > 1) {
            s_sum[par][wave] = sum;
            __syncthreads();
            sum = s_sum[par][wave - part];
            for (int i = 1; i < W; i++) sum += s_sum[par][wave - part + i];
        }
        const float f = (float)reciprocal_root(sum / (double)a.K + a.eps);
#pragma unroll
        for (int r = 0; r < R; r++) {
            Raw16<false> w;
            if constexpr (LW) {
#pragma unroll
                for (int i = 0; i < 4; i++) w.a[i] = *w_place(r, i);
            } else {
                w.load(wr, at[r]);
            }
            float wv[16];
            w.values(wv);
#pragma unroll
            for (int i = 0; i < 16; i++) v[r][i] = v[r][i] * f * (wv[i] + a.offset);
        }
        if (a.normed) {
            const int64_t bytes = a.K * (a.normed_bf16 ? 2 : 4);
            const __amdgpu_buffer_rsrc_t rn = row(a.normed, m, bytes, bytes);
#pragma unroll
            for (int r = 0; r < R; r++) store16(rn, at[r], a.normed_bf16, v[r]);
        }
        if (!a.x_q) continue;
        // as k_prepare_tokens has it
        float top = 0.0f;
#pragma unroll
        for (int r = 0; r < R; r++) {
            fwht256_row16(v[r], lane & 15);
#pragma unroll
            for (int i = 0; i < 16; i++) top = fmaxf(top, fabsf(v[r][i]));
        }
        top = wave_max(top);
        if (W > 1) {
            s_top[par][wave] = top;
            __syncthreads();
            top = s_top[par][wave - part];
            for (int i = 1; i < W; i++) top = fmaxf(top, s_top[par][wave - part + i]);
        }
        const float s = top / 127.0f, rs = s >= kQuantFastMin ? 1.0f / s : 0.0f;
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(s), row(a.s_x, m, 4, 4), part == 0 && lane == 0 ? 0u : kOutside, 0, 0);
        const __amdgpu_buffer_rsrc_t rq = row(a.x_q, m, a.K, a.K);
#pragma unroll
        for (int r = 0; r < R; r++) {
            const uint4 q = top > 0.0f ? quant16_auto(v[r], s, rs) : make_uint4(0, 0, 0, 0);
            __builtin_amdgcn_raw_buffer_store_b128(u32x4{q.x, q.y, q.z, q.w}, rq, at[r], 0, 0);
        }
    }
}

constexpr int kWavesPerCu = 16;  // tokens' waves on a compute unit: what the registers hold at R 3

template <bool XB, bool RB, int R, int kThreads>
hipError_t launch_r(const NormArgs &a, int W, int num_cu, hipStream_t stream) {
    // workgroups of four waves or one token
    const int waves = W >= 4 || W == 3 ? W : 4;
    const int64_t tokens = waves / W, need = (a.M + tokens - 1) / tokens;
    const int64_t most = kWavesPerCu / waves > 1 ? (int64_t)num_cu * (kWavesPerCu / waves) : num_cu;
    const unsigned grid = (unsigned)(need < most ? need : most);
    // weights in LDS where a workgroup has several tokens
    if constexpr (R <= 3) {
        if (256 * 16 * R * W <= kMaxWeights && need > most) {
            k_add_norm<XB, RB, R, kThreads, true><<<grid, 64 * waves, 0, stream>>>(a, W);
            return hipGetLastError();
        }
    }
    k_add_norm<XB, RB, R, kThreads, false><<<grid, 64 * waves, 0, stream>>>(a, W);
    return hipGetLastError();
}

// Blocks a group of 16 lanes (fp32 to bf16; 1, 2 and 3): 1 token of 5120 5.5, 5.0 and 6.2 us, 512 10.6, 9.3 and 9.5, 2048 29.3, 26.2 and
// 27.1, 8192 102, 89 and 79, where 2 and 3 leave as many places of a token's waves empty; 8192 x 4096 bf16 2 59 and 3
// 67, 3000 x 8192 47 and 56, where 3 leaves more; 16384 x 1024 bf16 1 32 and 2 37.  4 and 5 blocks in workgroups of 256 threads
// spill or have too few waves: 8192 x 5120 94 and 82 at best.
// 3 blocks of an fp32 residual spill 11 to 20 registers in the loop over tokens (of a bf16 one 4 at most), and gain less.  2 and 3, bf16 + bf16 /
// bf16 + fp32 / fp32 + fp32: 8192 x 5120 72 and 59 / 107 and 108 / 123 and 122, 4096 x 5120 38 and 32 / 48 and 48 / 55 and 64, 8192 x 2816
// 37 and 31 / 49 and 58 / 61 and 70, 8192 x 9216 137 and 116 / 219 and 200 / 251 and 221.
// K beyond 32768 needs 4 blocks in 1024 threads, 128 registers each, and spills 14 (fp32 + bf16), 42 (bf16 + bf16) and 77 to 81: 512 x 65536 77 us
// (3.9 TB/s), 81 (2.9), fp32 residuals 152 and 158 (2.4 and 2.8); 512 x 32768, 2 blocks, 4.1 to 4.7 TB/s.
template <bool XB, bool RB>
hipError_t launch_t(const NormArgs &a, int num_cu, hipStream_t stream) {
    const int64_t nblk = a.K / kRot;
    auto W = [&](int r) { return (int)((nblk + 4 * r - 1) / (4 * r)); };
    if (W(1) == 1) return launch_r<XB, RB, 1, 1024>(a, 1, num_cu, stream);
    if (W(2) > 16) return launch_r<XB, RB, 4, 1024>(a, W(4), num_cu, stream);
    if (a.M >= 4096 && W(3) <= 4 && 3 * W(3) <= 2 * W(2)) return launch_r<XB, RB, 3, 256>(a, W(3), num_cu, stream);
    return launch_r<XB, RB, 2, 1024>(a, W(2), num_cu, stream);
}

}  // namespace

hipError_t launch_add_norm(const NormArgs &a, int x_bf16, int r_bf16, int num_cu, hipStream_t stream) {
    if (x_bf16) return r_bf16 ? launch_t<true, true>(a, num_cu, stream) : launch_t<true, false>(a, num_cu, stream);
    return r_bf16 ? launch_t<false, true>(a, num_cu, stream) : launch_t<false, false>(a, num_cu, stream);
}

}  // namespace w4a8
