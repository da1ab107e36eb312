// C ABI of libw4a8_attn.so: argument validation, device check and dispatch of the attention
// operators.  The public contract is stated in include/w4a8_attn.h.
#include <math.h>
#include <string.h>

#include <atomic>

#include "attn_internal.h"

namespace {

constexpr int kMaxDevices = 64;
constexpr int64_t kInt31 = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxTokens = int64_t(1) << 24;  // a grid holds fewer than 2^32 threads
std::atomic<int> g_kind[kMaxDevices];  // 0 = unknown, 1 = gfx950, 2 = other
std::atomic<int> g_cus[kMaxDevices];

// The current device, which must be a gfx950.  Returns a w4a8_status.
int current_device(int *num_cu) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return W4A8_ERR_HIP;
    if (dev < 0 || dev >= kMaxDevices) return W4A8_ERR_DEVICE;
    int kind = g_kind[dev].load(std::memory_order_acquire);
    if (kind == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return W4A8_ERR_HIP;
        kind = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
        g_cus[dev].store(prop.multiProcessorCount, std::memory_order_relaxed);
        g_kind[dev].store(kind, std::memory_order_release);
    }
    if (kind != 1) return W4A8_ERR_DEVICE;
    *num_cu = g_cus[dev].load(std::memory_order_relaxed);
    return W4A8_OK;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool valid_dtype(int d) { return d == W4A8_F32 || d == W4A8_BF16; }
inline bool valid_dim(int d) { return d == 64 || d == 128 || d == 256; }

// log2 of a valid page size, or -1
inline int page_shift(int p) {
    for (int s = 4; s <= 8; s++)
        if (p == 1 << s) return s;
    return -1;
}

int check_cache(const w4a8_kv_cache *c, const w4a8_sequences *s) {
    if (!c || !s || !c->k || !c->v || !c->k_scale || !c->v_scale || !s->page_table || !s->cu_tokens || !s->seq_lens)
        return W4A8_ERR_NULL;
    if (c->num_pages < 1 || c->num_pages > kInt31 || c->kv_heads < 1 || c->kv_heads > 1024 ||
        page_shift(c->page_size) < 0 || !valid_dim(c->head_dim))
        return W4A8_ERR_SHAPE;
    if (s->B < 1 || s->B > 65536 || s->table_width < 1 || s->table_width > kInt31 / c->page_size) return W4A8_ERR_SHAPE;
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale) ||
        !aligned16(s->page_table) || !aligned16(s->cu_tokens) || !aligned16(s->seq_lens))
        return W4A8_ERR_ALIGN;
    return W4A8_OK;
}

// rows of `width` consecutive values, `stride` elements apart
inline bool valid_stride(int64_t stride, int64_t width) {
    return stride >= width && stride % 8 == 0 && stride <= (int64_t(1) << 31);
}

int check_heads(const w4a8_heads *h, int head_dim) {
    if (!h->x || !h->out) return W4A8_ERR_NULL;
    if (h->heads < 1 || !valid_stride(h->head_stride, head_dim) || h->token_stride < 0 || h->token_stride % 8 != 0 ||
        h->token_stride > (int64_t(1) << 40))
        return W4A8_ERR_SHAPE;
    if (!aligned16(h->x) || !aligned16(h->out) || !aligned16(h->weight)) return W4A8_ERR_ALIGN;
    return W4A8_OK;
}

inline int status_of(hipError_t e) { return e == hipSuccess ? W4A8_OK : W4A8_ERR_HIP; }

}  // namespace

extern "C" {

const char *w4a8_attn_status_string(int status) {
    switch (status) {
        case W4A8_OK: return "ok";
        case W4A8_ERR_NULL: return "a required pointer is NULL";
        case W4A8_ERR_SHAPE: return "a size, stride or number is out of its range";
        case W4A8_ERR_DTYPE: return "unknown dtype or scaling code";
        case W4A8_ERR_ALIGN: return "a pointer is not 16-byte aligned";
        case W4A8_ERR_WORKSPACE: return "workspace missing or too small";
        case W4A8_ERR_HIP: return "HIP runtime call or kernel launch failed";
        case W4A8_ERR_DEVICE: return "current device is not a gfx950 GPU";
        default: return "unknown status";
    }
}

int w4a8_rope_frequencies(int rotary_dim, double base, int scaling, double factor, double original_context,
                          double beta_fast, double beta_slow, double *inv_freq, float *attn_factor) {
    if (!inv_freq || !attn_factor) return W4A8_ERR_NULL;
    if (scaling < W4A8_ROPE_PLAIN || scaling > W4A8_ROPE_YARN) return W4A8_ERR_DTYPE;
    const int R = rotary_dim;
    // negated comparisons refuse NaN too
    if (R < 2 || R % 2 != 0 || !(base > 1.0) || !(base < INFINITY)) return W4A8_ERR_SHAPE;
    if (scaling != W4A8_ROPE_PLAIN && (!(factor >= 1.0) || !(factor < INFINITY))) return W4A8_ERR_SHAPE;
    if (scaling == W4A8_ROPE_NTK && R == 2) return W4A8_ERR_SHAPE;
    if (scaling == W4A8_ROPE_YARN && (!(original_context > 0.0) || !(original_context < INFINITY) ||
                                      !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !(beta_fast < INFINITY)))
        return W4A8_ERR_SHAPE;
    const double b = scaling == W4A8_ROPE_NTK ? base * pow(factor, R / (R - 2.0)) : base;
    double low = 0.0, high = 0.0;
    if (scaling == W4A8_ROPE_YARN) {
        const double turn = 2.0 * 3.14159265358979323846;
        low = floor(R * log(original_context / (turn * beta_fast)) / (2.0 * log(base)));
        high = ceil(R * log(original_context / (turn * beta_slow)) / (2.0 * log(base)));
        low = low > 0.0 ? low : 0.0;
        high = high < R - 1.0 ? high : R - 1.0;
    }
    for (int i = 0; i < R / 2; i++) {
        const double f = pow(b, -2.0 * i / R);
        if (scaling == W4A8_ROPE_LINEAR) {
            inv_freq[i] = f / factor;
        } else if (scaling == W4A8_ROPE_YARN) {
            const double width = high - low > 1e-3 ? high - low : 1e-3;
            double ramp = (i - low) / width;
            ramp = ramp < 0.0 ? 0.0 : ramp > 1.0 ? 1.0 : ramp;
            inv_freq[i] = f / factor * ramp + f * (1.0 - ramp);
        } else {
            inv_freq[i] = f;
        }
    }
    *attn_factor = scaling == W4A8_ROPE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
    return W4A8_OK;
}

int w4a8_qk_norm_rope(const w4a8_heads *q, const w4a8_heads *k, int64_t M, int head_dim, int x_dtype, int out_dtype,
                      const int32_t *positions, const double *inv_freq, int rotary_dim, int interleaved,
                      float attn_factor, float eps, float weight_offset, void *stream) {
    if (!q || !positions || !inv_freq) return W4A8_ERR_NULL;
    if (!valid_dim(head_dim)) return W4A8_ERR_SHAPE;
    int st = check_heads(q, head_dim);
    if (st == W4A8_OK && k) st = check_heads(k, head_dim);
    if (st != W4A8_OK) return st;
    const int64_t heads = (int64_t)q->heads + (k ? k->heads : 0);
    if (M < 1 || M > kMaxTokens || heads > 65536 || M > kInt31 / heads || rotary_dim < 16 || rotary_dim > head_dim ||
        rotary_dim % 16 != 0 || (interleaved != 0 && interleaved != 1) || !(eps >= 0.0f))
        return W4A8_ERR_SHAPE;
    if (!valid_dtype(x_dtype) || !valid_dtype(out_dtype)) return W4A8_ERR_DTYPE;
    if (!aligned16(positions) || !aligned16(inv_freq)) return W4A8_ERR_ALIGN;
    int num_cu = 0;
    st = current_device(&num_cu);
    if (st != W4A8_OK) return st;
    const w4a8_heads none{nullptr, 0, 0, 0, nullptr, nullptr};
    w4a8::RopeArgs a{*q, k ? *k : none, M, positions, inv_freq, rotary_dim, interleaved, attn_factor, eps, weight_offset};
    return status_of(w4a8::launch_qk_norm_rope(a, head_dim, x_dtype == W4A8_BF16, out_dtype == W4A8_BF16, num_cu,
                                               static_cast<hipStream_t>(stream)));
}

int w4a8_kv_append(const void *k, int64_t k_stride, const void *v, int64_t v_stride, int dtype, int64_t M,
                   const w4a8_kv_cache *cache, const w4a8_sequences *seqs, void *stream) {
    if (!k || !v) return W4A8_ERR_NULL;
    int st = check_cache(cache, seqs);
    if (st != W4A8_OK) return st;
    const int64_t width = (int64_t)cache->kv_heads * cache->head_dim;
    if (M < 1 || M > kMaxTokens || !valid_stride(k_stride, width) || !valid_stride(v_stride, width)) return W4A8_ERR_SHAPE;
    if (!valid_dtype(dtype)) return W4A8_ERR_DTYPE;
    if (!aligned16(k) || !aligned16(v)) return W4A8_ERR_ALIGN;
    int num_cu = 0;
    st = current_device(&num_cu);
    if (st != W4A8_OK) return st;
    w4a8::AppendArgs a{{k, v}, {k_stride, v_stride}, M, *cache, *seqs, page_shift(cache->page_size)};
    return status_of(w4a8::launch_kv_append(a, dtype == W4A8_BF16, static_cast<hipStream_t>(stream)));
}

// Rows (new tokens x query heads of a cache head) a sequence has on average decide the kernel:
// to 16 they are the split kernel's block of 16, to 64 its blocks of 32, above that the prompt kernel.
// Measured (us; 32 / 8 heads of 128, 16 sequences on 4000 tokens, bf16): 16 rows 34.6 in blocks of 16, 42.7 in blocks
// of 32; 20 rows 48.3 and 43.9.  On 2000 tokens, blocks of 32 and the prompt kernel: 32 rows 34.0 and 43.1, 64 rows
// 38.6 and 43.9, 96 rows 64.7 and 45.3.  24 / 4 heads of 256, 2 x 30000: 60 rows 89.5 and 94.0, 96 rows 129 and 98;
// fp32, 8 x 2000: 48 rows 35.3 and 37.0, 96 rows 52.7 and 39.9.
// The average is all that the host has, of the rows and sequences of the arguments: rows behind the last sequence and
// sequences without a token count.  A call of quite different sequences takes one kernel for all of them (24 / 4 heads of 256,
// in one call and in two): 63 x 1 token on 4000 and 2048 fresh ones 373 and 204 us, 63 x 1 and 512 on 4000 306 and 203, 255 x 1 on
// 1000 and 2000 fresh ones 471 and 217, 200 x 1 on 2000 and 256 fresh ones 187 and 199.  16 x 1 on 4000 is 37.0 us, with 48 rows behind
// them 42.3, with 240 78.3; 8 x 40 on 4000 is 90.4, with 56 empty sequences 103, 64 x 40 on 2000 183, with 192 empty ones 476.
constexpr int64_t kSplitRows = 64;
static int64_t rows_per_sequence(int64_t M, int64_t B, int group) { return (M * group + B - 1) / B; }

// The pieces of cut units that the kernel for this shape leaves behind the counters.
static int64_t attn_bytes(int64_t M, int64_t B, int group, int head_dim, int num_cu) {
    return w4a8::kAttnCounterBytes + (rows_per_sequence(M, B, group) <= kSplitRows ? w4a8::attn_split_bytes(head_dim, num_cu)
                                                                           : w4a8::attn_prompt_bytes(head_dim, num_cu));
}

static int check_attn_shape(int64_t M, int64_t B, int q_heads, int kv_heads, int head_dim) {
    if (B < 1 || B > 65536 || kv_heads < 1 || kv_heads > 1024 || !valid_dim(head_dim)) return W4A8_ERR_SHAPE;
    if (q_heads < 1 || q_heads > 8192 || q_heads % kv_heads != 0 || M < 1 || M > kMaxTokens ||
        M > kInt31 / q_heads)
        return W4A8_ERR_SHAPE;
    return W4A8_OK;
}

int64_t w4a8_kv_attention_workspace_bytes(int64_t M, int64_t B, int q_heads, int kv_heads, int head_dim) {
    int st = check_attn_shape(M, B, q_heads, kv_heads, head_dim);
    if (st != W4A8_OK) return -st;
    int num_cu = 0;
    st = current_device(&num_cu);
    if (st != W4A8_OK) return -st;
    // a call of fewer tokens or sequences may take either kernel
    const int64_t split = w4a8::attn_split_bytes(head_dim, num_cu), prompt = w4a8::attn_prompt_bytes(head_dim, num_cu);
    return w4a8::kAttnCounterBytes + (M * (q_heads / kv_heads) <= kSplitRows || split > prompt ? split : prompt);
}

int w4a8_kv_attention(const void *q, int64_t q_stride, int dtype, int64_t M, int q_heads, const w4a8_kv_cache *cache,
                      const w4a8_sequences *seqs, float sm_scale, int causal, int64_t window, void *o, void *workspace,
                      int64_t workspace_bytes, void *stream) {
    if (!q || !o) return W4A8_ERR_NULL;
    int st = check_cache(cache, seqs);
    if (st != W4A8_OK) return st;
    st = check_attn_shape(M, seqs->B, q_heads, cache->kv_heads, cache->head_dim);
    if (st != W4A8_OK) return st;
    if (!valid_stride(q_stride, (int64_t)q_heads * cache->head_dim) || (causal != 0 && causal != 1) || window < 0 ||
        (window > 0 && !causal) || !(sm_scale - sm_scale == 0.0f))
        return W4A8_ERR_SHAPE;
    if (!valid_dtype(dtype)) return W4A8_ERR_DTYPE;
    if (!aligned16(q) || !aligned16(o) || !aligned16(workspace)) return W4A8_ERR_ALIGN;
    int num_cu = 0;
    st = current_device(&num_cu);
    if (st != W4A8_OK) return st;
    const int group = q_heads / cache->kv_heads;
    if (!workspace || workspace_bytes < attn_bytes(M, seqs->B, group, cache->head_dim, num_cu)) return W4A8_ERR_WORKSPACE;
    // a counter for each workgroup of the widest launch
    if (2 * num_cu > w4a8::kAttnCounterBytes / 4) return W4A8_ERR_DEVICE;
    // a window that no length reaches is none
    if (window > kInt31) window = 0;
    w4a8::AttnArgs a{q, q_stride, M, q_heads, group, *cache, *seqs, page_shift(cache->page_size), sm_scale, causal, window, o,
                     workspace};
    hipStream_t st2 = static_cast<hipStream_t>(stream);
    const int64_t rows = rows_per_sequence(M, seqs->B, group);
    return status_of(rows <= kSplitRows ? w4a8::launch_attn_split(a, dtype == W4A8_BF16, rows <= 16 ? 1 : 2, num_cu, st2)
                                : w4a8::launch_attn_prompt(a, dtype == W4A8_BF16, num_cu, st2));
}

}  // extern "C"
