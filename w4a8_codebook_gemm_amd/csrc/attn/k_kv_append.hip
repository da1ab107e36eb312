// Append of keys and values into the int8 paged cache.
//
// A job is one page of one sequence that gets new tokens; a team of threads does one job for one
// head of keys or of values: the largest magnitude of its tokens, the page's scale, the
// earlier codes where the scale grew, the new codes.  A row of head_dim values is held by
// head_dim / 16 lanes, 16 consecutive values a lane: 32 or 64 bytes read, one 16-byte store.
// Up to 4 passes over the job's rows stay in registers between the maximum and the codes, as they
// lie in memory; longer jobs read their rows twice, the second time from L2.
//
// The team is one wave where that holds a page in its 4 passes (pages of 4096 / head_dim tokens or fewer) or
// where a sequence has 4 new tokens on average or fewer, and the workgroup elsewhere.  A workgroup a page was
// 16.7 us for 256 sequences x 1 token (8 heads of 128) and 59.5 us for 16384 tokens in pages of 16, mostly
// workgroups starting; a wave a page is 7.8 us and 30.2 us.  Pages of 64 at head_dim 128 take 15.5 us for
// 8 x 1024 tokens with a workgroup, and would read every row twice with a wave.
//
// Bound by HBM with long prompts: 2 or 4 bytes read and one written a value; bf16 3.4 TB/s over launches of 50 and of
// 100 MB (14 to 15 and 29 us), fp32 4.0 over 84 MB (18.5 to 21 us), where a copy runs at 4.75.  Some 4 us are the start,
// the rest is each team's chain: its page number is waited for before its tokens are asked for.  Bound by
// latency with single tokens: 4.5 us for 61 sequences, of them the chain of reads from the sequence to its
// page, the scale and the token.
//
// Which page a team has is found on the device, where the lengths are: every wave runs
// the sequences' page counts through a prefix sum, 64 at a time, until its job's is reached.  The waves are as many as the
// tokens, so this grows with the square of the sequences: one token each (2 heads of 128) is 21 us for 1024, 90 for 4096, 0.96 ms
// for 16384 and 13.5 ms for 65536.
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

// 16 values of a row as they lie in memory: a bf16 pair stays one register.
template <bool BF16>
struct Raw {
    static constexpr int kWords = BF16 ? 8 : 16;
    uint4 w[kWords / 4];
    __device__ __forceinline__ void load(const void *x, int64_t off) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(x) + off * (BF16 ? 2 : 4));
#pragma unroll
        for (int i = 0; i < kWords / 4; i++) w[i] = p[i];
    }
    __device__ __forceinline__ void values(float v[16]) const {
#pragma unroll
        for (int i = 0; i < kWords / 4; i++) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if constexpr (BF16) {
                    v[8 * i + 2 * j] = __uint_as_float(u[j] << 16);
                    v[8 * i + 2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
                } else {
                    v[4 * i + j] = __uint_as_float(u[j]);
                }
            }
        }
    }
    __device__ __forceinline__ float top() const {
        float v[16], t = 0.0f;
        values(v);
#pragma unroll
        for (int i = 0; i < 16; i++) t = fmaxf(t, fabsf(v[i]));
        return t;
    }
};

// TEAM threads (one wave, or the workgroup) have one page, head and side.
template <int D, bool BF16, int TEAM>
__global__ __launch_bounds__(kThreads) void k_kv_append(AppendArgs a) {
    constexpr int kLanes = D / 16;
    constexpr int kRows = TEAM / kLanes;  // rows a pass
    __shared__ float s_max[kThreads / 64];
    const int tid = threadIdx.x % TEAM;
    const int side = (int)((blockIdx.y * blockDim.x + threadIdx.x) / TEAM);
    if (side >= 2 * a.c.kv_heads) return;  // uniform over the team, as the next is
    const Job job = find_job(a, blockIdx.x);
    if (job.page < 0) return;
    const int head = side >> 1, kv = side & 1;
    const int64_t ph = (int64_t)job.page * a.c.kv_heads + head;
    float *scale = (kv ? a.c.v_scale : a.c.k_scale) + ph;
    int8_t *codes = (kv ? a.c.v : a.c.k) + ph * a.c.page_size * D;
    const int64_t x0 = job.row * a.stride[kv] + head * D + 16 * (tid % kLanes);
    const int r0 = tid / kLanes;
    const float before = job.slot ? *scale : 0.0f;

    Raw<BF16> keep[kKeep];
#pragma unroll
    for (int p = 0; p < kKeep; p++) {
        const int r = r0 + p * kRows;
        keep[p] = Raw<BF16>{};
        if (r < job.rows) keep[p].load(a.x[kv], x0 + r * a.stride[kv]);
    }
    float top = 0.0f;
#pragma unroll
    for (int p = 0; p < kKeep; p++) top = fmaxf(top, keep[p].top());
    for (int r = r0 + kKeep * kRows; r < job.rows; r += kRows) {
        Raw<BF16> x;
        x.load(a.x[kv], x0 + r * a.stride[kv]);
        top = fmaxf(top, x.top());
    }
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) top = fmaxf(top, __shfl_xor(top, s));
    if constexpr (TEAM > 64) {
        if ((tid & 63) == 0) s_max[tid >> 6] = top;
        __syncthreads();
        top = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
    }

    float s = top / 127.0f;
    if (before > 0.0f) {
        // the smallest j >= 0 with top <= room * 2^j, from the exponents and fractions
        // (127 times a scale may pass fp32's range: every finite value has room then)
        const float room = fminf(127.0f * before, 0x1.fffffep127f);
        int et = 0, er = 0;
        const float mt = frexpf(top, &et), mr = frexpf(room, &er);
        int j = top > 0.0f ? et - er + (mt > mr ? 1 : 0) : 0;
        j = j < 0 ? 0 : j;
        s = ldexpf(before, j);
        if (j > 0) {
            const float down = j < 20 ? ldexpf(1.0f, -j) : 0.0f;  // |code| 2^-8 < 1/2 already
            for (int i = tid; i < job.slot * (D / 4); i += TEAM) {
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
    auto put = [&](int r, const Raw<BF16> &x) {
        float v[16];
        x.values(v);
        *reinterpret_cast<uint4 *>(y + r * D) = s > 0.0f ? quant16_auto(v, s, inv) : make_uint4(0, 0, 0, 0);
    };
#pragma unroll
    for (int p = 0; p < kKeep; p++) {
        const int r = r0 + p * kRows;
        if constexpr (BF16) {
            // widened anew: the widened values kept from above would halve the waves a SIMD holds
#pragma unroll
            for (int i = 0; i < Raw<BF16>::kWords / 4; i++)
                asm("" : "+v"(keep[p].w[i].x), "+v"(keep[p].w[i].y), "+v"(keep[p].w[i].z), "+v"(keep[p].w[i].w));
        }
        if (r < job.rows) put(r, keep[p]);
    }
    for (int r = r0 + kKeep * kRows; r < job.rows; r += kRows) {
        Raw<BF16> x;
        x.load(a.x[kv], x0 + r * a.stride[kv]);
        put(r, x);
    }
    if (tid == 0) *scale = s;  // the team has read it: its value went into s
}

template <int D, int TEAM>
hipError_t launch_team(const AppendArgs &a, int bf16, int64_t jobs, hipStream_t stream) {
    const int sides = 2 * a.c.kv_heads;
    const int threads = sides * TEAM < kThreads ? sides * TEAM : kThreads;
    const dim3 grid((unsigned)jobs, (unsigned)((sides * TEAM + threads - 1) / threads));
    if (bf16)
        k_kv_append<D, true, TEAM><<<grid, threads, 0, stream>>>(a);
    else
        k_kv_append<D, false, TEAM><<<grid, threads, 0, stream>>>(a);
    return hipGetLastError();
}

template <int D>
hipError_t launch_d(const AppendArgs &a, int bf16, hipStream_t stream) {
    // pages a call can touch: a sequence's first and last may be partial
    int64_t jobs = (a.M >> a.page_shift) + 2 * a.s.B;
    if (jobs > a.M) jobs = a.M;
    const bool one_wave = a.c.page_size <= kKeep * 1024 / D || a.M <= 4 * a.s.B;
    return one_wave ? launch_team<D, 64>(a, bf16, jobs, stream) : launch_team<D, kThreads>(a, bf16, jobs, stream);
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
