// C ABI of libw4a8_serve.so: argument validation, device check and dispatch of the serving
// operators.  The public contract is stated in include/w4a8_serve.h.
#include <math.h>
#include <string.h>

#include <atomic>

#include "serve_internal.h"

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

// rows of `width` consecutive values, `stride` elements apart
inline bool valid_stride(int64_t stride, int64_t width) {
    return stride >= width && stride % 8 == 0 && stride <= (int64_t(1) << 31);
}

int check_pages(const w4a8_pages *p) {
    if (!p || !p->page_table || !p->seq_lens || !p->free_pages || !p->free_count) return W4A8_ERR_NULL;
    if (p->B < 1 || p->B > 65536 || page_shift(p->page_size) < 0 || p->table_width < 1 ||
        p->table_width > kInt31 / p->page_size || p->num_pages < 1 || p->num_pages > kInt31)
        return W4A8_ERR_SHAPE;
    if (!aligned16(p->page_table) || !aligned16(p->seq_lens) || !aligned16(p->free_pages) || !aligned16(p->free_count))
        return W4A8_ERR_ALIGN;
    return W4A8_OK;
}

int check_cache(const w4a8_kv4_cache *c) {
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || !c->k_unit || !c->v_unit) return W4A8_ERR_NULL;
    if (c->num_pages < 1 || c->num_pages > kInt31 || c->kv_heads < 1 || c->kv_heads > 1024 ||
        page_shift(c->page_size) < 0 || !valid_dim(c->head_dim))
        return W4A8_ERR_SHAPE;
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale) ||
        !aligned16(c->k_unit) || !aligned16(c->v_unit))
        return W4A8_ERR_ALIGN;
    return W4A8_OK;
}

int check_sequences(const w4a8_sequences *s, int page_size) {
    if (!s || !s->page_table || !s->cu_tokens || !s->seq_lens) return W4A8_ERR_NULL;
    if (s->B < 1 || s->B > 65536 || s->table_width < 1 || s->table_width > kInt31 / page_size) return W4A8_ERR_SHAPE;
    if (!aligned16(s->page_table) || !aligned16(s->cu_tokens) || !aligned16(s->seq_lens)) return W4A8_ERR_ALIGN;
    return W4A8_OK;
}

inline int status_of(hipError_t e) { return e == hipSuccess ? W4A8_OK : W4A8_ERR_HIP; }

}  // namespace

extern "C" {

const char *w4a8_serve_status_string(int status) {
    switch (status) {
        case W4A8_OK: return "ok";
        case W4A8_ERR_NULL: return "a required pointer is NULL";
        case W4A8_ERR_SHAPE: return "a size, stride or number is out of its range";
        case W4A8_ERR_DTYPE: return "unknown dtype code";
        case W4A8_ERR_ALIGN: return "a pointer is not 16-byte aligned";
        case W4A8_ERR_WORKSPACE: return "workspace missing or too small";
        case W4A8_ERR_HIP: return "HIP runtime call or kernel launch failed";
        case W4A8_ERR_DEVICE: return "current device is not a gfx950 GPU";
        default: return "unknown status";
    }
}

int w4a8_add_norm_prepare(const void *x, int x_dtype, int64_t x_stride, const void *r, int r_dtype, int64_t r_stride,
                          const float *weight, float weight_offset, float eps, int64_t M, int64_t K, void *h, void *normed,
                          int normed_dtype, int8_t *x_q, float *s_x, void *stream) {
    if (!x || !weight || !x_q != !s_x || (!x_q && !normed) || (h && !r)) return W4A8_ERR_NULL;
    if (M < 1 || M > kMaxTokens || K < 256 || K > 65536 || K % 256 != 0 || !valid_stride(x_stride, K) ||
        (r && !valid_stride(r_stride, K)) || !(eps >= 0.0f) || !(eps < INFINITY) || !(weight_offset - weight_offset == 0.0f))
        return W4A8_ERR_SHAPE;
    if (!valid_dtype(x_dtype) || (r && !valid_dtype(r_dtype)) || (normed && !valid_dtype(normed_dtype))) return W4A8_ERR_DTYPE;
    if (!aligned16(x) || !aligned16(r) || !aligned16(weight) || !aligned16(h) || !aligned16(normed) || !aligned16(x_q) ||
        !aligned16(s_x))
        return W4A8_ERR_ALIGN;
    int num_cu = 0;
    const int st = current_device(&num_cu);
    if (st != W4A8_OK) return st;
    const w4a8::NormArgs a{x, r, x_stride, r ? r_stride : K, weight, weight_offset, (double)eps, M, K, h, normed,
                           normed_dtype == W4A8_BF16, x_q, s_x};
    return status_of(w4a8::launch_add_norm(a, x_dtype == W4A8_BF16, r && r_dtype == W4A8_BF16, num_cu,
                                           static_cast<hipStream_t>(stream)));
}

int w4a8_pages_assign(const w4a8_pages *pages, const int32_t *new_tokens, int64_t M, const w4a8_batch *batch, void *stream) {
    int st = check_pages(pages);
    if (st != W4A8_OK) return st;
    if (!new_tokens || !batch || !batch->cu_tokens || !batch->seq_lens || !batch->positions || !batch->slots ||
        !batch->free_count || !batch->missing)
        return W4A8_ERR_NULL;
    if (M < 1 || M > kMaxTokens) return W4A8_ERR_SHAPE;
    if (!aligned16(new_tokens) || !aligned16(batch->cu_tokens) || !aligned16(batch->seq_lens) || !aligned16(batch->positions) ||
        !aligned16(batch->slots) || !aligned16(batch->free_count) || !aligned16(batch->missing))
        return W4A8_ERR_ALIGN;
    int num_cu = 0;
    st = current_device(&num_cu);
    if (st != W4A8_OK) return st;
    return status_of(w4a8::launch_pages_assign(*pages, page_shift(pages->page_size), new_tokens, M, *batch,
                                               static_cast<hipStream_t>(stream)));
}

int w4a8_pages_release(const w4a8_pages *pages, const int32_t *keep_lens, int32_t *seq_lens, int32_t *free_count,
                       void *stream) {
    int st = check_pages(pages);
    if (st != W4A8_OK) return st;
    if (!keep_lens || !seq_lens || !free_count) return W4A8_ERR_NULL;
    if (!aligned16(keep_lens) || !aligned16(seq_lens) || !aligned16(free_count)) return W4A8_ERR_ALIGN;
    int num_cu = 0;
    st = current_device(&num_cu);
    if (st != W4A8_OK) return st;
    return status_of(w4a8::launch_pages_release(*pages, page_shift(pages->page_size), keep_lens, seq_lens, free_count,
                                                static_cast<hipStream_t>(stream)));
}

int w4a8_kv4_append(const void *k, int64_t k_stride, const void *v, int64_t v_stride, int dtype, int64_t M,
                    const w4a8_kv4_cache *cache, const int64_t *slots, void *stream) {
    if (!k || !v || !slots) return W4A8_ERR_NULL;
    int st = check_cache(cache);
    if (st != W4A8_OK) return st;
    const int64_t width = (int64_t)cache->kv_heads * cache->head_dim;
    // (a wave takes 512 values of keys or of values; a grid holds fewer than 2^32 threads)
    if (M < 1 || M > kMaxTokens || (M + 15) * width > (int64_t(1) << 34) || !valid_stride(k_stride, width) ||
        !valid_stride(v_stride, width))
        return W4A8_ERR_SHAPE;
    if (!valid_dtype(dtype)) return W4A8_ERR_DTYPE;
    if (!aligned16(k) || !aligned16(v) || !aligned16(slots)) return W4A8_ERR_ALIGN;
    int num_cu = 0;
    st = current_device(&num_cu);
    if (st != W4A8_OK) return st;
    const w4a8::Append4Args a{{k, v}, {k_stride, v_stride}, M, *cache, slots, page_shift(cache->page_size)};
    return status_of(w4a8::launch_kv4_append(a, dtype == W4A8_BF16, static_cast<hipStream_t>(stream)));
}

// Rows (new tokens x query heads of a cache head) a sequence has on average decide the kernel: to kSplitRows the split
// kernel's, above that the prompt kernel's.  The average is all that the host has, of the rows and sequences of the arguments: rows
// behind the last sequence and sequences without a token count.  Split and prompt kernel (us; 16 sequences on 4000 tokens, 32 / 8
// heads of 128): 32 rows 35 and 57, 64 rows 46 and 58, 96 rows 75 and 59; 4 x 96 rows on 20k to 30k 133 and 90; 24 / 4 of 256, 48
// rows 59 and 71, 96 rows 88 and 73; fp32 of 64, 64 rows 29 and 34, 96 rows 43 and 35.
// A prompt's chunk among single tokens costs most: 63 tokens on 4000 with 512 on 4000 (24 / 4 of 256; 32 / 8 of 128) 212 and 144 us in
// one call, 169 and 127 in two; with 2048 fresh ones 377 and 342, 172 and 136 in two.
constexpr int64_t kSplitRows = 64;
static int64_t rows_per_sequence(int64_t M, int64_t B, int group) { return (M * group + B - 1) / B; }

// The pieces of cut units that the kernel for this shape leaves behind the counters.
static int64_t attn_bytes(int64_t M, int64_t B, int group, int head_dim, int num_cu) {
    return w4a8::kAttnCounterBytes + (rows_per_sequence(M, B, group) <= kSplitRows ? w4a8::kv4_split_bytes(head_dim, num_cu)
                                                                                 : w4a8::kv4_prompt_bytes(head_dim, num_cu));
}

static int check_attn_shape(int64_t M, int64_t B, int q_heads, int kv_heads, int head_dim) {
    if (B < 1 || B > 65536 || kv_heads < 1 || kv_heads > 1024 || !valid_dim(head_dim)) return W4A8_ERR_SHAPE;
    if (q_heads < 1 || q_heads > 8192 || q_heads % kv_heads != 0 || M < 1 || M > kMaxTokens || M > kInt31 / q_heads)
        return W4A8_ERR_SHAPE;
    return W4A8_OK;
}

int64_t w4a8_kv4_attention_workspace_bytes(int64_t M, int64_t B, int q_heads, int kv_heads, int head_dim) {
    int st = check_attn_shape(M, B, q_heads, kv_heads, head_dim);
    if (st != W4A8_OK) return -st;
    int num_cu = 0;
    st = current_device(&num_cu);
    if (st != W4A8_OK) return -st;
    // a call of fewer tokens or sequences may take either kernel
    const int64_t split = w4a8::kv4_split_bytes(head_dim, num_cu), prompt = w4a8::kv4_prompt_bytes(head_dim, num_cu);
    return w4a8::kAttnCounterBytes + (M * (q_heads / kv_heads) <= kSplitRows || split > prompt ? split : prompt);
}

int w4a8_kv4_attention(const void *q, int64_t q_stride, int dtype, int64_t M, int q_heads, const w4a8_kv4_cache *cache,
                       const w4a8_sequences *seqs, float sm_scale, int causal, int64_t window, void *o, void *workspace,
                       int64_t workspace_bytes, void *stream) {
    if (!q || !o) return W4A8_ERR_NULL;
    int st = check_cache(cache);
    if (st == W4A8_OK) st = check_sequences(seqs, cache->page_size);
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
    const w4a8::Attn4Args a{q, q_stride, M, q_heads, group, *cache, *seqs, page_shift(cache->page_size), sm_scale, causal, window, o,
                            workspace};
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t rows = rows_per_sequence(M, seqs->B, group);
    return status_of(rows <= kSplitRows ? w4a8::launch_kv4_split(a, dtype == W4A8_BF16, rows, num_cu, s)
                                        : w4a8::launch_kv4_prompt(a, dtype == W4A8_BF16, num_cu, s));
}

}  // extern "C"
