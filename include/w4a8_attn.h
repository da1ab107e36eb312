/*
 * w4a8_attn.h -- C ABI of the MI355X (gfx950) attention operators that stand between the
 * quantised projections of w4a8.h (libw4a8_attn.so): the norm of query and key heads with
 * their rotary positions, the append into an int8 paged cache, and attention over it.
 *
 * A decoder's attention layer runs as
 *   w4a8_forward_multi    x -> q, k, v                              (w4a8.h)
 *   w4a8_qk_norm_rope     q, k -> normed and rotated q, k
 *   w4a8_kv_append        k, v -> the cache's pages
 *   w4a8_kv_attention     q, cache -> o
 *   w4a8_forward          o -> the output projection                (w4a8.h)
 *
 * Conventions are those of w4a8.h: device pointers on the current HIP device, owned by the
 * caller and 16-byte aligned; no device memory is allocated; work is enqueued asynchronously
 * on `stream`; arguments are validated before anything is enqueued; status codes and dtype
 * codes are w4a8_status and w4a8_dtype; calls are re-entrant and thread-safe.  What lives in
 * device memory (positions, page tables, offsets, lengths) cannot be validated by the host:
 * the kernels read and write inside the given buffers whatever it holds.
 */
#ifndef W4A8_ATTN_H
#define W4A8_ATTN_H

#include "w4a8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Text of a status code as these entry points mean it (static storage; never NULL). */
W4A8_API const char *w4a8_attn_status_string(int status);

/* How rotary frequencies are stretched to contexts longer than the trained one. */
typedef enum {
    W4A8_ROPE_PLAIN = 0,   /* f_i = base^(-2 i / R) */
    W4A8_ROPE_LINEAR = 1,  /* f_i / factor */
    W4A8_ROPE_NTK = 2,     /* base * factor^(R / (R - 2)) in place of base (R > 2) */
    W4A8_ROPE_YARN = 3     /* by parts: f_i up to the index that turns beta_fast times in
                              original_context, f_i / factor from the one that turns beta_slow
                              times, a linear ramp between; attn_factor = 0.1 ln(factor) + 1 */
} w4a8_rope_scaling;

/*
 * The R / 2 rotary frequencies (radians a position, fp64) for w4a8_qk_norm_rope, written to
 * HOST memory, and the factor on cos and sin that goes with them (1 except for YARN).
 *  rotary_dim R >= 2, even;  base > 1;  factor >= 1 (ignored for PLAIN)
 *  original_context > 0, beta_fast > beta_slow > 0: read for YARN only.  The ramp's ends are
 *  i = R ln(original_context / (2 pi beta)) / (2 ln base), rounded down for beta_fast and up
 *  for beta_slow and held to [0, R - 1].
 * Returns W4A8_ERR_NULL, W4A8_ERR_SHAPE (a number out of its range) or W4A8_ERR_DTYPE (an
 * unknown scaling).  Touches no GPU.
 */
W4A8_API int w4a8_rope_frequencies(int rotary_dim, double base, int scaling, double factor, double original_context,
                                   double beta_fast, double beta_slow, double *inv_freq, float *attn_factor);

/* The heads of one projection for w4a8_qk_norm_rope. */
typedef struct {
    const void *x;         /* element (token m, head h, d) at x[m * token_stride + h * head_stride + d] */
    int64_t token_stride;  /* elements; strides are multiples of 8 elements */
    int64_t head_stride;   /* elements, at least head_dim */
    int heads;             /* >= 1 */
    const float *weight;   /* [head_dim] norm weights; NULL: no norm, rotation only */
    void *out;             /* [M][heads][head_dim], contiguous; may be x where layout and type are the same,
                              and overlaps nothing else of the call */
} w4a8_heads;

/*
 * Head norm and rotary positions of queries and keys in one pass, one launch:
 *   y = x * rsqrt(mean_d x^2 + eps) * (weight + weight_offset)         (y = x without weight)
 *   (a, b) -> (a c - b s, b c + a s),  c, s = attn_factor * cos, sin (position * inv_freq[i])
 * for the R / 2 pairs among the first R = rotary_dim values: (i, i + R/2), or (2 i, 2 i + 1)
 * when interleaved.  fp32 throughout, the angle reduced in fp64; one rounding, to out_dtype.
 *
 *  q, k          HOST structs; k may be NULL (queries only)
 *  head_dim      64, 128 or 256;  rotary_dim a multiple of 16 from 16 to head_dim
 *  positions     [M] int32, any value;  inv_freq  [R / 2] fp64, device memory
 *  x_dtype, out_dtype   of both projections;  weight_offset 1 for weights stored around zero
 *  1 <= M <= 2^24, (heads of q + k) <= 65536, M * heads < 2^31
 */
W4A8_API int w4a8_qk_norm_rope(const w4a8_heads *q, const w4a8_heads *k, int64_t M, int head_dim, int x_dtype,
                               int out_dtype, const int32_t *positions, const double *inv_freq, int rotary_dim,
                               int interleaved, float attn_factor, float eps, float weight_offset, void *stream);

/*
 * An int8 cache of keys and values in pages.  A page holds page_size consecutive tokens of
 * one sequence; for each of its heads it has the codes [page_size][head_dim] and one fp32
 * scale for keys and one for values (element = code * scale, codes -127..127; scales are finite
 * and not negative, as the append leaves them).
 */
typedef struct {
    int8_t *k, *v;            /* [num_pages][kv_heads][page_size][head_dim] */
    float *k_scale, *v_scale; /* [num_pages][kv_heads] */
    int64_t num_pages;        /* 1 .. 2^31 - 1 */
    int kv_heads;             /* 1 .. 1024 */
    int page_size;            /* 16, 32, 64, 128 or 256 */
    int head_dim;             /* 64, 128 or 256 */
} w4a8_kv_cache;

/*
 * The sequences of one call.  Sequence b's new tokens are rows cu_tokens[b] ..
 * cu_tokens[b + 1] - 1 (none is allowed); after the append it is seq_lens[b] tokens long, so
 * new token i has position seq_lens[b] - n + i.  Position t lives in page
 * page_table[b][t / page_size], slot t % page_size.  Entries past a sequence's last page are
 * not read.  Values outside their range are safe: offsets are held to [0, M], lengths to
 * [0, table_width * page_size], tokens in front of position 0 are dropped by the append and
 * see nothing, and the tokens of a page whose number is outside [0, num_pages) are neither
 * written nor seen (-1 marks a page that was given up).
 */
typedef struct {
    const int32_t *page_table; /* [B][table_width] */
    const int32_t *cu_tokens;  /* [B + 1], not decreasing */
    const int32_t *seq_lens;   /* [B] */
    int64_t B;                 /* 1 .. 65536 */
    int64_t table_width;       /* >= 1; table_width * page_size < 2^31 */
} w4a8_sequences;

/*
 * Append new keys and values to their sequences' pages.
 *   A page whose slot 0 is written (fresh): scale = max|x| / 127 over the tokens it gets.
 *   A page that holds earlier tokens: its scale grows by the smallest power of two 2^j, j >= 0,
 *   with max|x| <= fl32(127 scale) * 2^j, and the earlier codes become rint(code * 2^-j).  However
 *   often a page grows, an element is then off by at most one step of the final scale.
 *   (Earlier scale 0: scale = max|x| / 127.)
 *   code = clamp(rint(x / scale), -127, 127), IEEE division, ties to even; 0 where scale is 0.
 * Bit-exact and deterministic for finite values.  A NaN or an infinity leaves its page and head
 * without a meaning until slot 0 is written again, and no other page or head.  Slots behind the last
 * token keep their bytes.  A call must not append to a page twice,
 * from two sequences or at two places of one.  Its time grows with the square of the sequences beyond a few
 * thousand.
 *
 *  k, v   [M] tokens of kv_heads * head_dim consecutive values, k_stride and v_stride elements
 *         apart (multiples of 8, at least kv_heads * head_dim), element type dtype;  1 <= M <= 2^24
 */
W4A8_API int w4a8_kv_append(const void *k, int64_t k_stride, const void *v, int64_t v_stride, int dtype, int64_t M,
                            const w4a8_kv_cache *cache, const w4a8_sequences *seqs, void *stream);

/* What of a workspace has to be zero before its first use: its first bytes. */
#define W4A8_KV_ATTENTION_COUNTER_BYTES 8192

/*
 * Workspace bytes w4a8_kv_attention needs for up to M tokens and B sequences on the current
 * device (a negative status for an invalid shape).  Launches nothing.
 */
W4A8_API int64_t w4a8_kv_attention_workspace_bytes(int64_t M, int64_t B, int q_heads, int kv_heads, int head_dim);

/*
 * Attention of the new tokens' queries over the cache (the new keys appended before):
 *   o = sum_t p_t v_t,  p = softmax_t(sm_scale * q . k_t)
 * over the positions t that the query at position p sees: all of the sequence (causal 0), or
 * t <= p, and with window > 0 also t > p - window.  A query that sees nothing gives 0.  Query
 * head h reads cache head h / (q_heads / kv_heads).  Rows of o that belong to no sequence are
 * left as they were.  One kernel serves a call; which one goes by M * (q_heads / kv_heads) / B, the rows a
 * sequence has on average.  Any mix of sequences is right, but a batch of single tokens beside a long prompt
 * may take twice the time of two calls, and rows behind the last sequence or many sequences without a
 * token may choose the slower kernel.  Where a query is not finite, or a scale of a page that it sees is
 * negative or not finite, that row of o has no meaning; other rows, and rows that do not see the page, are
 * not touched by it.
 *
 *  q         [M] tokens of q_heads * head_dim consecutive values, q_stride elements apart (a
 *            multiple of 8), element type dtype;  1 <= M <= 2^24, M * q_heads < 2^31
 *  q_heads   a multiple of kv_heads, at most 8192
 *  causal    0 or 1;  window  0 (none) or >= 1, causal only
 *  o         [M][q_heads][head_dim], element type dtype; overlaps no other operand
 *  workspace device memory of w4a8_kv_attention_workspace_bytes(M, B, ...) bytes or more, its first
 *            W4A8_KV_ATTENTION_COUNTER_BYTES zero before its first use (the others may hold anything);
 *            every call that completes leaves these counters at zero, so one workspace serves later
 *            calls of any shape it is large enough for, one at a time: calls that may overlap need
 *            workspaces of their own.
 *
 * Scores, softmax statistics and sums are fp32: an exponent is off by some 2^-24 of the row's largest
 * |score|, so scores of 2^13 (in powers of two) cost a probability 2^-11 of itself.  bf16 queries are exact
 * in the products down to 2^-28 of a row's largest value.  With P the row's largest probability times value
 * scale, probabilities enter the second product as one fp16 number for bf16: off by 2^-11 of themselves, or by
 * 2^-33 P where they are below 2^-22 P; for fp32 as the sum of two: 2^-22 of themselves, 2^-37 P below 2^-15 P,
 * and fp32 queries likewise (2^-38 of the row's largest value below 2^-16 of it).  A score or a sum that
 * leaves fp32's range leaves the row without a meaning.  Deterministic.
 */
W4A8_API int w4a8_kv_attention(const void *q, int64_t q_stride, int dtype, int64_t M, int q_heads,
                               const w4a8_kv_cache *cache, const w4a8_sequences *seqs, float sm_scale, int causal,
                               int64_t window, void *o, void *workspace, int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A8_ATTN_H */
