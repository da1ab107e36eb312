/*
 * Host code of libw4a8_serve.so under AddressSanitizer and UndefinedBehaviorSanitizer (test
 * infrastructure only; tests/test_serving_sanitize.py builds serve_api.hip with host-side
 * sanitizers and runs this driver, no GPU needed).  Every entry point is called with invalid
 * arguments and must return its documented status before touching the GPU.  Prints "ok" and
 * exits 0 on success.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "w4a8_serve.h"

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

static int norm(int64_t xs, int64_t rs, int64_t M, int64_t K, float eps, int dt) {
    return w4a8_add_norm_prepare(FAKE, dt, xs, FAKE, dt, rs, FAKE, 0.0f, eps, M, K, FAKE, FAKE, dt, FAKE, FAKE, NULL);
}
static w4a8_pages pages(void) {
    w4a8_pages p = {FAKE, FAKE, FAKE, FAKE, 2, 4, 9, 16};
    return p;
}
static w4a8_batch batch(void) {
    w4a8_batch b = {FAKE, FAKE, FAKE, FAKE, FAKE, FAKE};
    return b;
}
static w4a8_kv4_cache cache(void) {
    w4a8_kv4_cache c = {FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 8, 4, 64, 128};
    return c;
}
static w4a8_sequences seqs(void) {
    w4a8_sequences s = {FAKE, FAKE, FAKE, 2, 4};
    return s;
}
static int append(const w4a8_kv4_cache *c, int64_t stride, int64_t M, const int64_t *slots) {
    return w4a8_kv4_append(FAKE, stride, FAKE, stride, W4A8_BF16, M, c, slots, NULL);
}
static int attn(const w4a8_kv4_cache *c, const w4a8_sequences *s, int64_t stride, int64_t M, int hq, float scale, int64_t window) {
    return w4a8_kv4_attention(FAKE, stride, W4A8_BF16, M, hq, c, s, scale, 1, window, FAKE, FAKE, INT64_MAX, NULL);
}

int main(void) {
    for (int i = -2; i < 12; i++)
        if (!w4a8_serve_status_string(i)) failures++;

    EXPECT(norm(512, 512, INT64_MAX, 512, 0.0f, W4A8_F32), W4A8_ERR_SHAPE);
    EXPECT(norm(512, 512, 1, INT64_MAX, 0.0f, W4A8_F32), W4A8_ERR_SHAPE);
    EXPECT(norm(512, 512, 1, INT64_MIN, 0.0f, W4A8_F32), W4A8_ERR_SHAPE);
    EXPECT(norm(INT64_MAX, 512, 1, 512, 0.0f, W4A8_F32), W4A8_ERR_SHAPE);
    EXPECT(norm(512, INT64_MIN, 1, 512, 0.0f, W4A8_F32), W4A8_ERR_SHAPE);
    EXPECT(norm(512, 512, 1, 512, NAN, W4A8_F32), W4A8_ERR_SHAPE);
    EXPECT(norm(512, 512, 1, 512, 0.0f, INT32_MAX), W4A8_ERR_DTYPE);
    EXPECT(w4a8_add_norm_prepare(FAKE, 0, 512, NULL, 77, INT64_MIN, FAKE, 0.0f, 0.0f, 1, 512, NULL, NULL, 77, NULL, NULL, NULL),
           W4A8_ERR_NULL);

    w4a8_pages p = pages();
    w4a8_batch b = batch();
    EXPECT(w4a8_pages_assign(NULL, FAKE, 1, &b, NULL), W4A8_ERR_NULL);
    EXPECT(w4a8_pages_assign(&p, FAKE, 1, NULL, NULL), W4A8_ERR_NULL);
    EXPECT(w4a8_pages_assign(&p, FAKE, INT64_MAX, &b, NULL), W4A8_ERR_SHAPE);
    EXPECT(w4a8_pages_assign(&p, FAKE, INT64_MIN, &b, NULL), W4A8_ERR_SHAPE);
    b.slots = MIS;
    EXPECT(w4a8_pages_assign(&p, FAKE, 1, &b, NULL), W4A8_ERR_ALIGN);
    EXPECT(w4a8_pages_release(&p, MIS, FAKE, FAKE, NULL), W4A8_ERR_ALIGN);
    EXPECT(w4a8_pages_release(&p, NULL, FAKE, FAKE, NULL), W4A8_ERR_NULL);
    p.page_size = INT32_MIN;
    EXPECT(w4a8_pages_release(&p, FAKE, FAKE, FAKE, NULL), W4A8_ERR_SHAPE);
    p = pages();
    p.table_width = INT64_MAX;
    EXPECT(w4a8_pages_release(&p, FAKE, FAKE, FAKE, NULL), W4A8_ERR_SHAPE);
    p = pages();
    p.num_pages = INT64_MAX;
    EXPECT(w4a8_pages_release(&p, FAKE, FAKE, FAKE, NULL), W4A8_ERR_SHAPE);
    p = pages();
    p.B = INT64_MIN;
    EXPECT(w4a8_pages_release(&p, FAKE, FAKE, FAKE, NULL), W4A8_ERR_SHAPE);

    w4a8_kv4_cache c = cache();
    w4a8_sequences s = seqs();
    EXPECT(append(NULL, 512, 1, FAKE), W4A8_ERR_NULL);
    EXPECT(append(&c, 512, 1, NULL), W4A8_ERR_NULL);
    EXPECT(append(&c, INT64_MAX, 1, FAKE), W4A8_ERR_SHAPE);
    EXPECT(append(&c, INT64_MIN, 1, FAKE), W4A8_ERR_SHAPE);
    EXPECT(append(&c, 512, INT64_MAX, FAKE), W4A8_ERR_SHAPE);
    EXPECT(append(&c, 512, INT64_MIN, FAKE), W4A8_ERR_SHAPE);
    EXPECT(attn(&c, NULL, 1024, 1, 8, 1.0f, 0), W4A8_ERR_NULL);
    EXPECT(attn(&c, &s, 1024, INT64_MAX, 8, 1.0f, 0), W4A8_ERR_SHAPE);
    EXPECT(attn(&c, &s, 1024, 1, INT32_MIN, 1.0f, 0), W4A8_ERR_SHAPE);
    EXPECT(attn(&c, &s, 1024, 1, 8, INFINITY, 0), W4A8_ERR_SHAPE);
    EXPECT(attn(&c, &s, 1024, 1, 8, 1.0f, INT64_MIN), W4A8_ERR_SHAPE);
    c.num_pages = INT64_MAX;
    EXPECT(append(&c, 512, 1, FAKE), W4A8_ERR_SHAPE);
    c = cache();
    c.page_size = INT32_MIN;
    EXPECT(attn(&c, &s, 1024, 1, 8, 1.0f, 0), W4A8_ERR_SHAPE);
    c = cache();
    s.table_width = INT64_MAX;
    EXPECT(attn(&c, &s, 1024, 1, 8, 1.0f, 0), W4A8_ERR_SHAPE);
    s = seqs();
    s.B = INT64_MAX;
    EXPECT(attn(&c, &s, 1024, 1, 8, 1.0f, 0), W4A8_ERR_SHAPE);
    EXPECT(w4a8_kv4_attention_workspace_bytes(INT64_MAX, 1, 8, 4, 128), -W4A8_ERR_SHAPE);
    EXPECT(w4a8_kv4_attention_workspace_bytes(1, INT64_MIN, 8, 4, 128), -W4A8_ERR_SHAPE);
    EXPECT(w4a8_kv4_attention_workspace_bytes(1, 1, 8, 0, 128), -W4A8_ERR_SHAPE);

    if (failures) return 1;
    puts("ok");
    return 0;
}
