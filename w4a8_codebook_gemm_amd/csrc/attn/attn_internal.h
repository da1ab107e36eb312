// Internal declarations of libw4a8_attn.so: launchers and the device helpers its kernels
// share.  Not part of the public ABI (include/w4a8_attn.h).
#pragma once

#include "../../../include/w4a8_attn.h"
#include "../w4a8_internal.h"

namespace w4a8 {

struct RopeArgs {
    w4a8_heads q, k;  // k.heads 0 where there are no keys
    int64_t M;
    const int32_t *positions;
    const double *inv_freq;
    int rotary;
    int interleaved;
    float attn_factor, eps, offset;
};
hipError_t launch_qk_norm_rope(const RopeArgs &a, int head_dim, int x_bf16, int out_bf16, int num_cu, hipStream_t stream);

struct AppendArgs {
    const void *x[2];    // keys, values
    int64_t stride[2];
    int64_t M;
    w4a8_kv_cache c;
    w4a8_sequences s;
    int page_shift;
};
hipError_t launch_kv_append(const AppendArgs &a, int bf16, hipStream_t stream);

struct AttnArgs {
    const void *q;
    int64_t q_stride;
    int64_t M;
    int hq, group;       // query heads, query heads for each cache head
    w4a8_kv_cache c;
    w4a8_sequences s;
    int page_shift;
    float scale;
    int causal;
    int64_t window;      // 0: none
    void *o;
    void *ws;
};
constexpr int64_t kAttnCounterBytes = W4A8_KV_ATTENTION_COUNTER_BYTES;  // arrival counters at the workspace's start
// Few rows a sequence: blocks of 16 (blocks 1) or 32 (2) rows.
int64_t attn_split_bytes(int head_dim, int num_cu);
hipError_t launch_attn_split(const AttnArgs &a, int bf16, int blocks, int num_cu, hipStream_t stream);
// Many rows a sequence.
int64_t attn_prompt_bytes(int head_dim, int num_cu);
hipError_t launch_attn_prompt(const AttnArgs &a, int bf16, int num_cu, hipStream_t stream);

// Two values as bf16, to nearest even (one instruction on gfx950).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    const bf16x2_t v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

// One sequence as the kernels see it, every number held to its range: rows first .. first + n - 1,
// length, and the position of the first row (negative where the length is shorter than n).
struct Seq {
    int64_t first;
    int n, len, pos0;
};
__device__ __forceinline__ Seq load_seq(const w4a8_sequences &s, int64_t M, int page_shift, int64_t b) {
    Seq q;
    const int64_t c0 = s.cu_tokens[b], c1 = s.cu_tokens[b + 1];
    q.first = c0 < 0 ? 0 : c0 > M ? M : c0;
    const int64_t last = c1 < q.first ? q.first : c1 > M ? M : c1;
    q.n = (int)(last - q.first);
    const int64_t most = s.table_width << page_shift;
    const int64_t len = s.seq_lens[b];
    q.len = (int)(len < 0 ? 0 : len > most ? most : len);
    q.pos0 = q.len - q.n;
    return q;
}

}  // namespace w4a8
