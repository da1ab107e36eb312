// Attention over the int8 paged cache: one wave for each query head of each token.
//
//   o = sum_t p_t v_t, p = softmax(scale q . k_t): one pass over the visible positions with the
// running maximum and sum, fp32 throughout.  Each lane holds head_dim / 64 values.
#include "attn_internal.h"

namespace w4a8 {
namespace {

template <int D, bool BF16>
__global__ __launch_bounds__(256) void k_attention(AttnArgs a) {
    constexpr int E = D / 64;
    const int lane = threadIdx.x & 63;
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (item >= a.M * a.hq) return;
    const int64_t m = item / a.hq;
    const int h = (int)(item % a.hq), kvh = h / a.group;
    // the last sequence that begins at or before the row
    int64_t lo = 0, hi = a.s.B;
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) / 2;
        if (a.s.cu_tokens[mid] <= m) lo = mid; else hi = mid;
    }
    const Seq q = load_seq(a.s, a.M, a.page_shift, lo);
    if (m < q.first || m >= q.first + q.n) return;
    const int pos = q.pos0 + (int)(m - q.first);
    const int end = a.causal ? pos + 1 : q.len;
    int64_t begin = a.window ? (int64_t)pos - a.window + 1 : 0;
    if (begin < 0) begin = 0;
    float x[E], acc[E], mx = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < E; i++) {
        const int64_t off = m * a.q_stride + h * D + lane * E + i;
        x[i] = (BF16 ? bf16_to_f32(static_cast<const uint16_t *>(a.q)[off]) : static_cast<const float *>(a.q)[off]) * a.scale;
        acc[i] = 0.0f;
    }
    for (int t = (int)begin; t < end; t++) {
        const int page = a.s.page_table[lo * a.s.table_width + (t >> a.page_shift)];
        if (page < 0 || page >= a.c.num_pages) continue;
        const int64_t ph = (int64_t)page * a.c.kv_heads + kvh;
        const int64_t off = (ph * a.c.page_size + (t & (a.c.page_size - 1))) * D + lane * E;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < E; i++) s = fmaf(x[i], (float)a.c.k[off + i], s);
#pragma unroll
        for (int w = 1; w < 64; w <<= 1) s += __shfl_xor(s, w);
        s *= a.c.k_scale[ph];
        const float top = fmaxf(mx, s), old = expf(mx - top), p = expf(s - top);
        const float pv = p * a.c.v_scale[ph];
        mx = top;
        sum = fmaf(sum, old, p);
#pragma unroll
        for (int i = 0; i < E; i++) acc[i] = fmaf(acc[i], old, pv * (float)a.c.v[off + i]);
    }
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int i = 0; i < E; i++) {
        const int64_t off = (m * a.hq + h) * D + lane * E + i;
        if (BF16) static_cast<uint16_t *>(a.o)[off] = f32_to_bf16_rne(acc[i] * inv);
        else static_cast<float *>(a.o)[off] = acc[i] * inv;
    }
}

template <int D>
hipError_t launch_d(const AttnArgs &a, int bf16, hipStream_t stream) {
    const unsigned grid = (unsigned)((a.M * a.hq + 3) / 4);
    if (bf16) k_attention<D, true><<<grid, 256, 0, stream>>>(a);
    else k_attention<D, false><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

int64_t attn_workspace_bytes(int64_t, int64_t, int, int, int, int) { return 0; }

hipError_t launch_kv_attention(const AttnArgs &a, int bf16, int, hipStream_t stream) {
    switch (a.c.head_dim) {
        case 64: return launch_d<64>(a, bf16, stream);
        case 128: return launch_d<128>(a, bf16, stream);
        default: return launch_d<256>(a, bf16, stream);
    }
}

}  // namespace w4a8
