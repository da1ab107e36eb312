// Internal declarations of libw4a8_serve.so: launchers and what its kernels share.  Not part of
// the public ABI (include/w4a8_serve.h).
#pragma once

#include "../../../include/w4a8_serve.h"
#include "../attn/attn_internal.h"

namespace w4a8 {

struct NormArgs {
    const void *x, *r;
    int64_t x_stride, r_stride;
    const float *w;
    float offset;
    double eps;
    int64_t M, K;
    void *h, *normed;
    int normed_bf16;
    int8_t *x_q;
    float *s_x;
};
hipError_t launch_add_norm(const NormArgs &a, int x_bf16, int r_bf16, int num_cu, hipStream_t stream);

hipError_t launch_pages_assign(const w4a8_pages &p, int page_shift, const int32_t *new_tokens, int64_t M,
                               const w4a8_batch &out, hipStream_t stream);
hipError_t launch_pages_release(const w4a8_pages &p, int page_shift, const int32_t *keep, int32_t *lens, int32_t *count,
                                hipStream_t stream);

struct Append4Args {
    const void *x[2];    // keys, values
    int64_t stride[2];
    int64_t M;
    w4a8_kv4_cache c;
    const int64_t *slots;
    int page_shift;
};
hipError_t launch_kv4_append(const Append4Args &a, int bf16, hipStream_t stream);

struct Attn4Args {
    const void *q;
    int64_t q_stride;
    int64_t M;
    int hq, group;       // query heads, query heads for each cache head
    w4a8_kv4_cache c;
    w4a8_sequences s;
    int page_shift;
    float scale;
    int causal;
    int64_t window;      // 0: none
    void *o;
    void *ws;
};
static_assert(W4A8_KV4_ATTENTION_COUNTER_BYTES == kAttnCounterBytes, "one counter area for both caches");
// Few rows a sequence (on average).
int64_t kv4_split_bytes(int head_dim, int num_cu);
hipError_t launch_kv4_split(const Attn4Args &a, int bf16, int64_t rows, int num_cu, hipStream_t stream);
// Many rows a sequence.
int64_t kv4_prompt_bytes(int head_dim, int num_cu);
hipError_t launch_kv4_prompt(const Attn4Args &a, int bf16, int num_cu, hipStream_t stream);

}  // namespace w4a8
