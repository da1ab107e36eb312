/*
 * Host code of libw4a8_attn.so under AddressSanitizer and UndefinedBehaviorSanitizer (test
 * infrastructure only; tests/test_attention_sanitize.py builds attn_api.hip with host-side
 * sanitizers and runs this driver, no GPU needed).  Every entry point is called with invalid
 * arguments and must return its documented status before touching the GPU; the host-only
 * calls run in full.  Prints "ok" and exits 0 on success.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "w4a8_attn.h"

#define FAKE ((void *)(uintptr_t)0x10000) /* 16-byte aligned, never dereferenced */
#define MIS ((void *)(uintptr_t)0x10008)  /* misaligned */

static int failures = 0;
#define EXPECT(call, want)                                                                        \
    do {                                                                                          \
        const long long got_ = (long long)(call);                                                 \
        if (got_ != (long long)(want)) {                                                          \
            fprintf(stderr, "line %d: %s returned %lld, expected %lld\n", __LINE__, #call, got_,  \
                    (long long)(want));                                                           \
            failures++;                                                                           \
        }                                                                                         \
    } while (0)

static w4a8_heads heads(void) {
    w4a8_heads h = {FAKE, 1024, 128, 8, NULL, FAKE};
    return h;
}
static int rope(const w4a8_heads *q, const w4a8_heads *k, int64_t M, int rotary, float eps, int xdt) {
    return w4a8_qk_norm_rope(q, k, M, 128, xdt, W4A8_BF16, FAKE, FAKE, rotary, 0, 1.0f, eps, 0.0f, NULL);
}

static w4a8_kv_cache cache(void) {
    w4a8_kv_cache c = {FAKE, FAKE, FAKE, FAKE, 8, 4, 64, 128};
    return c;
}
static w4a8_sequences seqs(void) {
    w4a8_sequences s = {FAKE, FAKE, FAKE, 2, 4};
    return s;
}
static int append(const w4a8_kv_cache *c, const w4a8_sequences *s, int64_t stride, int64_t M) {
    return w4a8_kv_append(FAKE, stride, FAKE, stride, W4A8_BF16, M, c, s, NULL);
}
static int attn(const w4a8_kv_cache *c, const w4a8_sequences *s, int64_t stride, int64_t M, int hq, float scale, int64_t window) {
    return w4a8_kv_attention(FAKE, stride, W4A8_BF16, M, hq, c, s, scale, 1, window, FAKE, FAKE, INT64_MAX, NULL);
}

int main(void) {
    for (int i = -2; i < 12; i++)
        if (!w4a8_attn_status_string(i)) failures++;

    double f[128];
    float attn_factor;
    const int kinds[] = {W4A8_ROPE_PLAIN, W4A8_ROPE_LINEAR, W4A8_ROPE_NTK, W4A8_ROPE_YARN};
    for (int i = 0; i < 4; i++)
        for (int r = 4; r <= 256; r *= 2) {
            EXPECT(w4a8_rope_frequencies(r, 1e6, kinds[i], 1e30, 1e-30, 1e30, 1e-30, f, &attn_factor), W4A8_OK);
            EXPECT(w4a8_rope_frequencies(r, 1.0 + 1e-15, kinds[i], 1.0, 1e300, 32.0, 1.0, f, &attn_factor), W4A8_OK);
        }
    EXPECT(w4a8_rope_frequencies(64, 1e6, 4, 1.0, 1.0, 2.0, 1.0, f, &attn_factor), W4A8_ERR_DTYPE);
    EXPECT(w4a8_rope_frequencies(INT32_MIN, 1e6, 0, 1.0, 1.0, 2.0, 1.0, f, &attn_factor), W4A8_ERR_SHAPE);
    EXPECT(w4a8_rope_frequencies(64, NAN, 0, 1.0, 1.0, 2.0, 1.0, f, &attn_factor), W4A8_ERR_SHAPE);
    EXPECT(w4a8_rope_frequencies(64, 1e6, 0, 1.0, 1.0, 2.0, 1.0, NULL, &attn_factor), W4A8_ERR_NULL);

    w4a8_heads q = heads(), k = heads();
    EXPECT(rope(NULL, &k, 1, 64, 0.0f, W4A8_BF16), W4A8_ERR_NULL);
    EXPECT(rope(&q, &k, INT64_MAX, 64, 0.0f, W4A8_BF16), W4A8_ERR_SHAPE);
    EXPECT(rope(&q, &k, 1, INT32_MAX, 0.0f, W4A8_BF16), W4A8_ERR_SHAPE);
    EXPECT(rope(&q, NULL, 1, 64, -1.0f, W4A8_BF16), W4A8_ERR_SHAPE);
    EXPECT(rope(&q, &k, 1, 64, 0.0f, INT32_MAX), W4A8_ERR_DTYPE);
    k.heads = INT32_MAX;
    EXPECT(rope(&q, &k, 1, 64, 0.0f, W4A8_BF16), W4A8_ERR_SHAPE);
    k = heads();
    k.token_stride = INT64_MAX - 7;
    EXPECT(rope(&q, &k, 1, 64, 0.0f, W4A8_BF16), W4A8_ERR_SHAPE);
    k = heads();
    k.head_stride = INT64_MIN;
    EXPECT(rope(&q, &k, 1, 64, 0.0f, W4A8_BF16), W4A8_ERR_SHAPE);
    k = heads();
    k.out = MIS;
    EXPECT(rope(&q, &k, 1, 64, 0.0f, W4A8_BF16), W4A8_ERR_ALIGN);

    w4a8_kv_cache c = cache();
    w4a8_sequences s = seqs();
    EXPECT(append(NULL, &s, 512, 1), W4A8_ERR_NULL);
    EXPECT(append(&c, NULL, 512, 1), W4A8_ERR_NULL);
    EXPECT(append(&c, &s, INT64_MAX, 1), W4A8_ERR_SHAPE);
    EXPECT(append(&c, &s, INT64_MIN, 1), W4A8_ERR_SHAPE);
    EXPECT(append(&c, &s, 512, INT64_MIN), W4A8_ERR_SHAPE);
    EXPECT(attn(&c, &s, 1024, INT64_MAX, 8, 1.0f, 0), W4A8_ERR_SHAPE);
    EXPECT(attn(&c, &s, 1024, 1, INT32_MIN, 1.0f, 0), W4A8_ERR_SHAPE);
    EXPECT(attn(&c, &s, 1024, 1, 8, INFINITY, 0), W4A8_ERR_SHAPE);
    EXPECT(attn(&c, &s, 1024, 1, 8, 1.0f, INT64_MIN), W4A8_ERR_SHAPE);
    c.num_pages = INT64_MAX;
    EXPECT(append(&c, &s, 512, 1), W4A8_ERR_SHAPE);
    c = cache();
    c.page_size = INT32_MIN;
    EXPECT(attn(&c, &s, 1024, 1, 8, 1.0f, 0), W4A8_ERR_SHAPE);
    c = cache();
    s.table_width = INT64_MAX;
    EXPECT(attn(&c, &s, 1024, 1, 8, 1.0f, 0), W4A8_ERR_SHAPE);
    s = seqs();
    s.B = INT64_MAX;
    EXPECT(append(&c, &s, 512, 1), W4A8_ERR_SHAPE);
    EXPECT(w4a8_kv_attention_workspace_bytes(INT64_MAX, 1, 8, 4, 128), -W4A8_ERR_SHAPE);
    EXPECT(w4a8_kv_attention_workspace_bytes(1, INT64_MIN, 8, 4, 128), -W4A8_ERR_SHAPE);
    EXPECT(w4a8_kv_attention_workspace_bytes(1, 1, 8, 0, 128), -W4A8_ERR_SHAPE);

    if (failures) return 1;
    puts("ok");
    return 0;
}
