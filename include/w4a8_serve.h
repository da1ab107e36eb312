/*
 * w4a8_serve.h -- C ABI of the MI355X (gfx950) serving operators that stand around the quantised
 * products of w4a8.h and beside the attention operators of w4a8_attn.h (libw4a8_serve.so): the
 * residual's addition with its norm and the products' int8 input, pages taken and given back on
 * the GPU, and a paged cache held in 4 bits with the attention over it.
 *
 * A decode step runs as
 *   w4a8_pages_assign       lengths, new tokens -> page table, offsets, positions, slots
 *   then for each layer
 *   w4a8_add_norm_prepare   output of the layer before, residual -> residual, x_q, s_x
 *   w4a8_linear_multi       x_q, s_x -> q, k, v                                        (w4a8.h)
 *   w4a8_qk_norm_rope       q, k, positions -> normed and rotated q, k                 (w4a8_attn.h)
 *   w4a8_kv4_append         k, v, slots -> the cache's pages
 *   w4a8_kv4_attention      q, cache -> o
 *   w4a8_forward            o -> the output projection                                 (w4a8.h)
 *   w4a8_add_norm_prepare, and the MLP's products
 *   and w4a8_pages_release  for what ended or was refused.
 *
 * Conventions are those of w4a8.h: device pointers on the current HIP device, owned by the
 * caller and 16-byte aligned; no device memory is allocated; work is enqueued asynchronously
 * on `stream`; arguments are validated before anything is enqueued; status codes and dtype
 * codes are w4a8_status and w4a8_dtype; calls are re-entrant and thread-safe.  What lives in
 * device memory (page tables, lengths, lists of free pages, slots) cannot be validated by the
 * host: the kernels read and write inside the given buffers whatever it holds.
 */
#ifndef W4A8_SERVE_H
#define W4A8_SERVE_H

#include "w4a8_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Text of a status code as these entry points mean it (static storage; never NULL). */
W4A8_API const char *w4a8_serve_status_string(int status);

/*
 * The residual's addition, the RMS norm and the quantised products' input in one pass, one launch:
 *   h = x + r                          fp32, rounded to r's type
 *   f = fl32(1 / sqrt(mean h^2 + eps))  of the rounded h; the mean and the root in fp64
 *   y = fl32(fl32(h f) fl32(weight + weight_offset))
 *   x_q, s_x = what w4a8_prepare_activation gives for y: each block of 256 rotated, one scale a token
 *
 *  x          [M] rows of K consecutive values, x_stride elements apart (a multiple of 8, at least K), type x_dtype
 *  r          [M] rows likewise, type r_dtype; NULL: no residual, h is x (r_dtype and r_stride are not read)
 *  weight     [K] fp32;  weight_offset 1 for weights stored around zero;  eps >= 0, finite
 *  h          [M][K], type r_dtype; may be r or x where layout and type are the same; NULL: not kept (so without r)
 *  normed     [M][K] y rounded to normed_dtype, for layers that are not quantised; NULL: not wanted
 *  x_q, s_x   [M][K] int8, [M] fp32, for w4a8_linear and w4a8_linear_multi; both NULL: not wanted (then normed is)
 *  1 <= M <= 2^24;  256 <= K <= 65536, K % 256 == 0
 *
 * Outputs overlap no other operand but h as stated.  Bit-exact and deterministic but for the fp64
 * sum's last bits: f is off by one fp32 step where they decide its rounding, one row in some 2^28.  Values that are not finite, and
 * rows of zeros with eps 0, leave their row without a meaning and no other.
 */
W4A8_API int w4a8_add_norm_prepare(const void *x, int x_dtype, int64_t x_stride, const void *r, int r_dtype,
                                   int64_t r_stride, const float *weight, float weight_offset, float eps, int64_t M,
                                   int64_t K, void *h, void *normed, int normed_dtype, int8_t *x_q, float *s_x,
                                   void *stream);

/*
 * The pages of B sequences and those that are free.  Position t of sequence b lives in page
 * page_table[b][t / page_size], as in w4a8_sequences; a page belongs to one sequence.  Lengths outside
 * [0, table_width * page_size] and counts outside [0, num_pages] are held to that range.
 */
typedef struct {
    int32_t *page_table;  /* [B][table_width] */
    int32_t *seq_lens;    /* [B] */
    int32_t *free_pages;  /* [num_pages]: numbers of the free pages; the last one is handed out first */
    int32_t *free_count;  /* [1]: how many of them there are */
    int64_t B;            /* 1 .. 65536 */
    int64_t table_width;  /* >= 1; table_width * page_size < 2^31 */
    int64_t num_pages;    /* 1 .. 2^31 - 1 */
    int page_size;        /* 16, 32, 64, 128 or 256 */
} w4a8_pages;

/* What w4a8_pages_assign says of a step's new tokens. */
typedef struct {
    int32_t *cu_tokens;   /* [B + 1] */
    int32_t *seq_lens;    /* [B]: lengths with the new tokens; may be the pages' own */
    int32_t *positions;   /* [M] */
    int64_t *slots;       /* [M]: page * page_size + place in it */
    int32_t *free_count;  /* [1]; may be the pages' own */
    int32_t *missing;     /* [1]: pages that the list, or a sequence's table, had no room for */
} w4a8_batch;

/*
 * Room for a step's new tokens: sequence b grows from seq_lens[b] by new_tokens[b] (held to 0 or more).
 * Pages come off the list's end in order of sequences and positions; where it has run out the table
 * gets -1, which the append drops and attention does not see.  Tokens behind a sequence's table are
 * counted in cu_tokens, their slot is -1, and the length is held to the table (the sequence's rows have
 * no meaning then, others do).  Rows are numbered 0 .. M - 1: offsets are held to M, and sequences whose
 * tokens would lie behind it grow by the rows that there are.  Rows behind the last token get position 0 and slot -1.
 * The free list itself is not changed, only its count: with outputs apart from the pages' own lengths and
 * count, the call can be repeated.  Deterministic.  One launch; two where lengths or count are written in place and M
 * is beyond a few thousand.  Every workgroup walks all sequences.
 *  new_tokens  [B] int32;  1 <= M <= 2^24
 */
W4A8_API int w4a8_pages_assign(const w4a8_pages *pages, const int32_t *new_tokens, int64_t M, const w4a8_batch *batch,
                               void *stream);

/*
 * Pages given back: sequence b keeps its first keep_lens[b] tokens (0: it ended; held to 0 .. its length).
 * The pages behind go to the list's end, the last one of the last sequence first, so that assigning the same tokens
 * again hands out the same pages; entries outside [0, num_pages) (pages that were missing, or given up) are
 * passed over, and so is what the list has no room for.  The table's entries stay as they are.  One workgroup.
 *  keep_lens  [B] int32
 *  seq_lens, free_count   the new lengths [B] and count [1]; may be the pages' own
 */
W4A8_API int w4a8_pages_release(const w4a8_pages *pages, const int32_t *keep_lens, int32_t *seq_lens, int32_t *free_count,
                                void *stream);

/*
 * A cache of keys and values in pages, in 4 bits (4.5 with the scales).  16 consecutive values of a token's
 * head share a scale byte b:
 *   value = e2m1(code) * sc(b) * unit[head]
 *   e2m1  0, 0.5, 1, 1.5, 2, 3, 4, 6 for the codes 0 .. 7, the same negative for 8 .. 15
 *   sc(b) = b for b < 16, else (16 + b % 16) * 2^(b / 16 - 1):  0 .. 507904, five significant bits
 * so a head's largest magnitude is 3047424 units, and groups whose largest is under 96 units lose precision.
 * The unit 2^-14 (186 at most, 0.006) suits normed keys and most values.  Two codes a byte, the first one low.
 * Every byte is a valid code and a valid scale.
 */
typedef struct {
    uint8_t *k, *v;               /* codes [num_pages][kv_heads][page_size][head_dim / 2] */
    uint8_t *k_scale;             /* [num_pages][kv_heads][page_size][head_dim / 16] */
    uint8_t *v_scale;             /* [num_pages][kv_heads][head_dim / 16][page_size] */
    const float *k_unit, *v_unit; /* [kv_heads], 2^-120 .. 2^100 */
    int64_t num_pages;            /* 1 .. 2^31 - 1 */
    int kv_heads;                 /* 1 .. 1024 */
    int page_size;                /* 16, 32, 64, 128 or 256 */
    int head_dim;                 /* 64, 128 or 256 */
} w4a8_kv4_cache;

/*
 * New keys and values into their slots (page * page_size + place, as w4a8_pages_assign gives them; slots
 * outside the cache, -1 among them, are dropped).  With t = max|x| / fl32(6 unit) over a group of 16, in fp32:
 *   b    = the nearest of 1 .. 255 to t by sc(b), ties to even
 *   code = the nearest to fl32(x / fl32(sc(b) unit)), ties to the even code, +-6 beyond; a zero keeps its sign
 * IEEE division throughout.  S = sc(b) unit is within 2^-5 of max|x| / 6 where that is 16 units or more, up to 507904.  In groups whose
 * max|x| is more than 15 units and at most 3047424, values are off by S / 4 at most up to 2 S, S / 2 up to 4 S and S beyond (and by
 * what fp32 division moves a border).  Smaller groups have no finer scales: there values are off by as much, or by 3 units (a group
 * whose largest is 8.9 units has S 1 and is cut to 6).  What is beyond 3047424 units is cut to it.  Bit-exact and deterministic; tokens
 * do not depend on one another.  A NaN leaves its value without a meaning; an infinity is the largest magnitude, and costs its
 * group's others theirs.
 * Two tokens of a call must not have the same slot.
 *
 *  k, v   [M] tokens of kv_heads * head_dim consecutive values, k_stride and v_stride elements
 *         apart (multiples of 8, at least kv_heads * head_dim), element type dtype;  1 <= M <= 2^24
 *  slots  [M] int64
 */
W4A8_API int w4a8_kv4_append(const void *k, int64_t k_stride, const void *v, int64_t v_stride, int dtype, int64_t M,
                             const w4a8_kv4_cache *cache, const int64_t *slots, void *stream);

/* What of a workspace has to be zero before its first use: its first bytes. */
#define W4A8_KV4_ATTENTION_COUNTER_BYTES 8192

/*
 * Workspace bytes w4a8_kv4_attention needs for up to M tokens and B sequences on the current
 * device (a negative status for an invalid shape).  Launches nothing.
 */
W4A8_API int64_t w4a8_kv4_attention_workspace_bytes(int64_t M, int64_t B, int q_heads, int kv_heads, int head_dim);

/*
 * Attention of the new tokens' queries over a cache in 4 bits: w4a8_kv_attention's operator, arguments
 * and rules (w4a8_attn.h), on w4a8_kv4_cache.
 *   o = sum_t p_t v_t,  p = softmax_t(sm_scale * q . k_t)
 * over the positions t that the query at position p sees: all of the sequence (causal 0), or
 * t <= p, and with window > 0 also t > p - window.  A query that sees nothing gives 0; pages outside
 * [0, num_pages) are not seen.  Query head h reads cache head h / (q_heads / kv_heads).  Rows of o that
 * belong to no sequence are left as they were.  Which kernel serves a call goes by M * (q_heads / kv_heads) / B, the
 * rows a sequence has on average; any mix of sequences is right, but a prompt among many single tokens is
 * faster in a call of its own.  A query that is not finite leaves its own row
 * without a meaning, a unit outside its range its head's.
 *
 *  q         [M] tokens of q_heads * head_dim consecutive values, q_stride elements apart (a
 *            multiple of 8), element type dtype;  1 <= M <= 2^24, M * q_heads < 2^31
 *  q_heads   a multiple of kv_heads, at most 8192
 *  causal    0 or 1;  window  0 (none) or >= 1, causal only
 *  o         [M][q_heads][head_dim], element type dtype; overlaps no other operand
 *  workspace device memory of w4a8_kv4_attention_workspace_bytes(M, B, ...) bytes or more, its first
 *            W4A8_KV4_ATTENTION_COUNTER_BYTES zero before its first use (the others may hold anything);
 *            every call that completes leaves these counters at zero, so one workspace serves later
 *            calls of any shape it is large enough for, one at a time: calls that may overlap need
 *            workspaces of their own.
 *
 * Cached values are exact in both products.  Scores, softmax statistics and sums are fp32: an exponent is off by
 * some 2^-24 of the row's largest |score| (in powers of two; from 2^26 on a row has no meaning).  bf16 queries are exact
 * in the products down to 2^-28 of a row's largest value, fp32 queries to 2^-22 of themselves (2^-38 of the row's largest
 * value below 2^-16 of it).  With P the row's largest probability so far, probabilities enter the second product as one
 * fp16 number for bf16: off by 2^-11 of themselves, or by 2^-35 P where they are below 2^-24 P; for fp32 as the sum of
 * two: 2^-22 of themselves, 2^-35 P below 2^-13 P; the parts of P grow by 2^(2^-22 |score|) with scores beyond 2^20.  A sum
 * that leaves fp32's range leaves the row without a meaning.  Deterministic.
 */
W4A8_API int w4a8_kv4_attention(const void *q, int64_t q_stride, int dtype, int64_t M, int q_heads,
                                const w4a8_kv4_cache *cache, const w4a8_sequences *seqs, float sm_scale, int causal,
                                int64_t window, void *o, void *workspace, int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A8_SERVE_H */
