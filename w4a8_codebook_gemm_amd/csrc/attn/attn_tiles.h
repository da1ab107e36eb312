// What the attention kernels share: operand fragments of v_mfma_f32_16x16x32_f16 made from
// int8 codes, queries as fp16, and the running softmax in powers of two.
#pragma once

#include "attn_internal.h"

namespace w4a8 {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kSign4 = 0x80808080u;  // code ^ 0x80 = code + 128, four at a time

// Eight consecutive codes (two dwords) as fp16, exact: the byte code + 128 under the exponent
// byte 0x64 is the fp16 number 1024 + 128 + code.
__device__ __forceinline__ half8_t codes_natural(uint32_t w0, uint32_t w1) {
    const half2_t bias = {(_Float16)1152.0f, (_Float16)1152.0f};
    uint32_t r[4];
    const uint32_t w[2] = {w0 ^ kSign4, w1 ^ kSign4};
#pragma unroll
    for (int i = 0; i < 2; i++) {
        r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, w[i], 0x04010400u)) - bias);
        r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, w[i], 0x04030402u)) - bias);
    }
    return __builtin_bit_cast(half8_t, make_uint4(r[0], r[1], r[2], r[3]));
}

// Byte J of two tokens' dwords (already ^ kSign4) as two fp16 numbers code * 2^-9, exact: the
// byte code + 128 alone is the subnormal (code + 128) 2^-24, which one packed multiply-add takes to
// 2^15 of it less 128 * 2^-9.  Picking the bytes and turning token rows into a fragment of
// consecutive tokens are the same permute.  (Subnormal operands themselves cost the matrix core's
// sums precision: next to weights of a wide range 16 bits of the largest product are left, not 22.)
template <int J>
__device__ __forceinline__ uint32_t codes_pair(uint32_t first, uint32_t second) {
    const half2_t up = {(_Float16)32768.0f, (_Float16)32768.0f}, bias = {(_Float16)-0.25f, (_Float16)-0.25f};
    const uint32_t u = __builtin_amdgcn_perm(second, first, 0x0C000C00u | (uint32_t)J | (uint32_t)(4 + J) << 16);
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(half2_t, u), up, bias));
}
constexpr int kCodeExp = 9;    // codes_pair's values are code * 2^-kCodeExp
constexpr int kProbExp = 14;   // probabilities enter the second product as p * 2^kProbExp

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    const half2_t h = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, h);
}

// 2^x for a whole-numbered x <= 0 of any size (0 below fp32's range).
__device__ __forceinline__ float pow2_down(float x) { return __builtin_amdgcn_exp2f(x); }

constexpr int kZeroExp = -300;       // exponent of a value scale of zero
constexpr float kLow = -3.0e38f;  // "no score yet"

// Eight consecutive query values as they lie in memory, and as fp32.
template <bool BF16>
struct RawQ {
    uint4 a, b;  // b: fp32 only
    __device__ __forceinline__ void load(const void *q, int64_t off) {
        if constexpr (BF16) {
            a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(q) + off);
        } else {
            const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(q) + off);
            a = p[0];
            b = p[1];
        }
    }
    __device__ __forceinline__ void values(float v[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
        if constexpr (BF16) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        } else {
            const uint32_t x[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                v[i] = __uint_as_float(w[i]);
                v[4 + i] = __uint_as_float(x[i]);
            }
        }
    }
};

// The larger of x and that of lane ^ 32 or lane ^ 16: with both operands x, the swap of half waves
// (of the odd 16-lane rows with the even ones) leaves the two in its two results.
typedef uint32_t uintx2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ float max_xor32(float x) {
    const uintx2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max_xor16(float x) {
    const uintx2 r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// x, as a value the compiler works from anew: what hangs on it is not kept in registers across a loop.
__device__ __forceinline__ int fresh(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// Lane l's value (l uniform) as a uniform one.
__device__ __forceinline__ int lane_value(int x, int l) { return __builtin_amdgcn_readlane(x, l); }
__device__ __forceinline__ int64_t lane_value(int64_t x, int l) {
    return (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)x, l) | (int64_t)__builtin_amdgcn_readlane((int)(x >> 32), l) << 32;
}

// Inclusive prefix sum over the wave's lanes: shifts within rows of 16, then the rows' ends to the rows after.
template <int kCtrl, int kRows>
__device__ __forceinline__ int64_t moved64(int64_t x) {
    const int lo = __builtin_amdgcn_update_dpp(0, (int)x, kCtrl, kRows, 0xF, false);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(x >> 32), kCtrl, kRows, 0xF, false);
    return (int64_t)(uint32_t)lo | (int64_t)hi << 32;
}
__device__ __forceinline__ int64_t scan64(int64_t x) {
    x += moved64<0x111, 0xF>(x);  // row_shr:1, 2, 4, 8
    x += moved64<0x112, 0xF>(x);
    x += moved64<0x114, 0xF>(x);
    x += moved64<0x118, 0xF>(x);
    x += moved64<0x142, 0xA>(x);  // row_bcast:15, 31
    x += moved64<0x143, 0xC>(x);
    return x;
}

// Tiles of T positions in front of position `to` >= 0.  Lengths end below 2^31: a signed sum would pass it.
template <int T>
__device__ __forceinline__ int tiles_to(int to) {
    return (int)(((uint32_t)to + (T - 1)) / T);
}

// a / b for a >= 0, b > 0
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
    return a / b;
}

// Four values of a piece, which other workgroups read or wrote, past the per-XCD caches: `off` bytes from a
// base that is uniform over the wave, in 16-byte accesses at device scope (cache bit sc1).
typedef uint32_t uintx4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ __amdgpu_buffer_rsrc_t shared_piece(const float *base, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void *)base, (short)0, bytes, 0x00020000);
}
__device__ __forceinline__ void put_shared4(__amdgpu_buffer_rsrc_t r, int off, float a, float b, float c, float d) {
    const uintx4 v = {__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d)};
    __builtin_amdgcn_raw_buffer_store_b128(v, r, off, 0, 16);
}
__device__ __forceinline__ floatx4 get_shared4(__amdgpu_buffer_rsrc_t r, int off) {
    return __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 16));
}

// How the line of tiles is cut.  A unit lies on it with `over` places in front of its tiles, what starting
// and joining it costs, and workgroup w's part begins at place w line / used.  A beginning among a
// unit's first `over` places is moved to the unit's, one less than `tail` places before its end
// to its end: what is left inside a unit is a cut, at the tile that lies there.
struct Line {
    int64_t length, used;
    int over, tail;
    __device__ __forceinline__ int64_t begin(int64_t w) const { return div64(w * length, used); }
    // this part [at, t1) of the unit of `tiles` tiles at u0, which begins at or before `at`: its tiles
    // from .. to - 1; false where it has none
    __device__ __forceinline__ bool part(int64_t at, int64_t t1, int64_t u0, int64_t u1, int tiles, int &from, int &to) const {
        from = 0;
        to = tiles;
        if (at > u0 + over) {
            if (at > u1 - tail) return false;
            from = (int)(at - u0 - over);
        }
        if (t1 < u1) {
            if (t1 <= u0 + over) return false;
            if (t1 <= u1 - tail && t1 - u0 - over < tiles) to = (int)(t1 - u0 - over);
        }
        return true;
    }
    // the workgroups that have pieces of the unit [u0, u1)
    __device__ __forceinline__ int64_t first(int64_t u0) const { return div64((u0 + over + 1) * used + length - 1, length) - 1; }
    __device__ __forceinline__ int64_t last(int64_t u1) const { return div64((u1 - tail + 1) * used - 1, length); }
};

// A running softmax: maximum m, exponent E of the weighted sum, sum L of the probabilities.  Joining
// two of them returns the factors for their weighted sums.
struct State {
    float m, E, L;
};
__device__ __forceinline__ State join(const State &a, const State &b, float &qa, float &qb) {
    State s;
    s.m = fmaxf(a.m, b.m);
    const float da = a.m - s.m, db = b.m - s.m;
    s.E = fmaxf(a.E + da, b.E + db);
    s.L = a.L * pow2_down(da) + b.L * pow2_down(db);
    qa = pow2_down(da + (a.E - s.E));
    qb = pow2_down(db + (b.E - s.E));
    return s;
}

// The pieces of a cut unit are joined in a tree, kRadix at a node: a workgroup leaves what it holds
// in the slot of its first piece and counts its arrival at the node; the last to arrive joins the
// node's slots in order of position and goes on a level up.  The sums do not depend on the order
// of arrival.  A node counts at the workgroup of its second child's first piece, which is no other
// node's, and its count ends at zero.  put(p) leaves this workgroup's part in piece p's slot;
// take(p, step, n) takes up the n slots p, p + step, ...  True for the workgroup that ends with the
// whole unit.
template <int kRadix, class Put, class Take>
__device__ __forceinline__ bool join_pieces(uint32_t *counters, int64_t w_first, int64_t w, int64_t w_end, int *s_flag, Put put, Take take) {
    const unsigned parts = (unsigned)(w_end - w_first + 1);
    unsigned lo = (unsigned)(w - w_first);
    for (unsigned size = 1; size < parts; size *= kRadix) {
        const unsigned node = lo / (size * kRadix) * (size * kRadix);
        unsigned n = (parts - node + size - 1) / size;  // children
        if (n > kRadix) n = kRadix;
        if (n == 1) continue;
        put(lo);
        // every store has left before the arrival is counted
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (threadIdx.x == 0) *s_flag = atomicInc(counters + w_first + node + size, n - 1) == n - 1;
        __syncthreads();
        const bool last = *s_flag;
        __syncthreads();
        if (!last) return false;
        take(node, size, n);
        lo = node;
    }
    return true;
}

// The positions [from, to) that new token i of a sequence sees: none in front of position 0.  Both ends
// grow with i, so a block's first token has the least of them and its last token the greatest.
__device__ __forceinline__ void sees(const AttnArgs &a, const Seq &q, int64_t i, int &from, int &to) {
    const int64_t pos = q.pos0 + i;
    const int64_t f = a.window ? pos - a.window + 1 : 0;
    from = f > 0 ? (int)f : 0;
    to = pos < 0 ? 0 : a.causal ? (int)(pos + 1) : q.len;
}

}  // namespace w4a8
