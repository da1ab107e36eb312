// Append of keys and values into the int8 paged cache.
//
// A job is one page of one sequence that gets new tokens; a workgroup does one job for one
// head of keys or of values: the largest magnitude of its tokens, the page's scale, the
// earlier codes where the scale grew, the new codes.  HBM bound (2 or 4 bytes read and one
// written a value) with long prompts, latency bound with single tokens.  A row of
// head_dim values is held by head_dim / 16 lanes, 16 consecutive values a lane: 32 or 64
// bytes read, one 16-byte store.  Up to 4 passes over the job's rows (64 rows at head_dim 256,
// 256 at 64) stay in registers between the maximum and the codes; longer jobs read their rows
// twice, the second time from L2.
//
// Which page a workgroup has is found on the device, where the lengths are: every wave runs
// the sequences' page counts through a prefix sum, 64 at a time, until its job's is reached.
#include "attn_internal.h"

namespace w4a8 {
namespace {

constexpr int kThreads = 256;
constexpr int kKeep = 4;  // passes held in registers

struct Job {
    int64_t row;   // first row of k / v
    int rows;      // tokens of the page
    int page;      // page number, -1: none
    int slot;      // first slot
};

__device__ __forceinline__ Job find_job(const AppendArgs &a, int64_t job) {
    const int lane = threadIdx.x & 63;
    Job out{0, 0, -1, 0};
    int64_t base = 0;
    for (int64_t b0 = 0; b0 < a.s.B; b0 += 64) {
        Seq q{0, 0, 0, 0};
        if (b0 + lane < a.s.B) q = load_seq(a.s, a.M, a.page_shift, b0 + lane);
        const int p0 = q.pos0 < 0 ? 0 : q.pos0;  // first position written
        const int j0 = p0 >> a.page_shift;
        const int cnt = q.n > 0 && q.len > p0 ? ((q.len - 1) >> a.page_shift) - j0 + 1 : 0;
        int incl = cnt;
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) {
            const int o = __shfl_up(incl, s);
            if (lane >= s) incl += o;
        }
        const int total = __shfl(incl, 63);
        if (job < base + total) {
            const int at = (int)(job - base);
            const uint64_t hit = __ballot(at >= incl - cnt && at < incl);
            const int src = __ffsll((unsigned long long)hit) - 1;
            const int j = __shfl(j0, src) + at - __shfl(incl - cnt, src);
            const int len = __shfl(q.len, src), first_pos = __shfl(p0, src), pos0 = __shfl(q.pos0, src);
            const int64_t first = __shfl((long long)q.first, src);
            const int from = j << a.page_shift > first_pos ? j << a.page_shift : first_pos;
            const int64_t page_end = (int64_t)(j + 1) << a.page_shift;
            const int to = page_end < len ? (int)page_end : len;
            const int page = a.s.page_table[(b0 + src) * a.s.table_width + j];
            out.row = first + (from - pos0);
            out.rows = to - from;
            out.slot = from & (a.c.page_size - 1);
            out.page = page >= 0 && page < a.c.num_pages ? page : -1;
            return out;
        }
        base += total;
    }
    return out;
}

template <int D, bool BF16>
__global__ __launch_bounds__(kThreads) void k_kv_append(AppendArgs a) {
    constexpr int kLanes = D / 16;
    constexpr int kRows = kThreads / kLanes;  // rows a pass
    __shared__ float s_max[kThreads / 64];
    const int tid = threadIdx.x;
    const Job job = find_job(a, blockIdx.x);
    if (job.page < 0) return;  // uniform over the workgroup
    const int head = blockIdx.y, kv = blockIdx.z;
    const int64_t ph = (int64_t)job.page * a.c.kv_heads + head;
    float *scale = (kv ? a.c.v_scale : a.c.k_scale) + ph;
    int8_t *codes = (kv ? a.c.v : a.c.k) + ph * a.c.page_size * D;
    const int64_t x0 = job.row * a.stride[kv] + head * D + 16 * (tid % kLanes);
    const int r0 = tid / kLanes;
    const float before = job.slot ? *scale : 0.0f;

    float keep[kKeep][16];
    float top = 0.0f;
#pragma unroll
    for (int p = 0; p < kKeep; p++) {
        const int r = r0 + p * kRows;
        if (r < job.rows) {
            load16<BF16>(a.x[kv], x0 + r * a.stride[kv], keep[p]);
#pragma unroll
            for (int i = 0; i < 16; i++) top = fmaxf(top, fabsf(keep[p][i]));
        }
    }
    for (int r = r0 + kKeep * kRows; r < job.rows; r += kRows) {
        float v[16];
        load16<BF16>(a.x[kv], x0 + r * a.stride[kv], v);
#pragma unroll
        for (int i = 0; i < 16; i++) top = fmaxf(top, fabsf(v[i]));
    }
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) top = fmaxf(top, __shfl_xor(top, s));
    if ((tid & 63) == 0) s_max[tid >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));

    float s = top / 127.0f;
    if (before > 0.0f) {
        // the smallest j >= 0 with top <= room * 2^j, from the exponents and fractions
        const float room = 127.0f * before;
        int et = 0, er = 0;
        const float mt = frexpf(top, &et), mr = frexpf(room, &er);
        int j = top > 0.0f ? et - er + (mt > mr ? 1 : 0) : 0;
        j = j < 0 ? 0 : j;
        s = ldexpf(before, j);
        if (j > 0) {
            const float down = j < 20 ? ldexpf(1.0f, -j) : 0.0f;  // |code| 2^-8 < 1/2 already
            for (int i = tid; i < job.slot * (D / 4); i += kThreads) {
                const uint32_t w = reinterpret_cast<const uint32_t *>(codes)[i];
                uint32_t u = 0;
#pragma unroll
                for (int q = 0; q < 4; q++)
                    u |= ((uint32_t)(int32_t)rintf((float)(int8_t)(w >> 8 * q) * down) & 0xFFu) << 8 * q;
                reinterpret_cast<uint32_t *>(codes)[i] = u;
            }
        }
    }
    // 1 / s is read by the corrected quotient only for scales that are far from underflow
    const float inv = 1.0f / s;
    int8_t *y = codes + (int64_t)job.slot * D + 16 * (tid % kLanes);
    auto put = [&](int r, const float v[16]) {
        *reinterpret_cast<uint4 *>(y + r * D) = s > 0.0f ? quant16_auto(v, s, inv) : make_uint4(0, 0, 0, 0);
    };
#pragma unroll
    for (int p = 0; p < kKeep; p++) {
        const int r = r0 + p * kRows;
        if (r < job.rows) put(r, keep[p]);
    }
    for (int r = r0 + kKeep * kRows; r < job.rows; r += kRows) {
        float v[16];
        load16<BF16>(a.x[kv], x0 + r * a.stride[kv], v);
        put(r, v);
    }
    if (tid == 0) *scale = s;  // every thread's read of it is before the barrier above
}

template <int D>
hipError_t launch_d(const AppendArgs &a, int bf16, hipStream_t stream) {
    // pages a call can touch: a sequence's first and last may be partial
    int64_t jobs = (a.M >> a.page_shift) + 2 * a.s.B;
    if (jobs > a.M) jobs = a.M;
    const dim3 grid((unsigned)jobs, (unsigned)a.c.kv_heads, 2);
    if (bf16)
        k_kv_append<D, true><<<grid, kThreads, 0, stream>>>(a);
    else
        k_kv_append<D, false><<<grid, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs &a, int bf16, hipStream_t stream) {
    switch (a.c.head_dim) {
        case 64: return launch_d<64>(a, bf16, stream);
        case 128: return launch_d<128>(a, bf16, stream);
        default: return launch_d<256>(a, bf16, stream);
    }
}

}  // namespace w4a8
