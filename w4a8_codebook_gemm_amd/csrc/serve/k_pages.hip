// Pages of sequences taken from and given back to a list on the device.
//
// Latency bound: a step's numbers are a few kilobytes.  A workgroup takes 1024 sequences at a time, one a
// thread: prefix sums of their new tokens and new pages, left in LDS, then every token and every
// page finds its sequence there by bisection.  With more tokens than a workgroup's threads care for, each of
// many workgroups walks all sequences and takes its share of each 1024's tokens and pages; what such a
// launch reads it must not write, so lengths and count that are updated in place are a second launch's.
//
// Measured: 61 sequences of a token 3.9 us, 700 with 138,000 tokens 4.8, 1021 with 260,000 5.1; 1024 sequences more are some 2.4 us
// more (16384 40, 65536 153).
#include "serve_internal.h"
#include "../attn/attn_tiles.h"

namespace w4a8 {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
// Tokens for which one workgroup is enough where lengths or count are written in place, which takes many a second launch: 8 x 250
// tokens 3.8 us, many 6.4, 8 x 500 4.8 and 6.3, 8 x 1000 6.7 and 6.4, 256 x 16 6.6 and 6.9.  Apart 8 x 250 tokens take one 4.5 us and
// many 3.9, 8 x 500 5.7 and 3.9, 256 x 16 6.2 and 4.1.
constexpr int kAlone = 4096;
// Entries of a thread at a time in giving back.  2, 4 and 8: 231 pages of 61 sequences 3.0, 3.5 and 4.3 us, 3347 of 256 4.2, 4.3 and 5.5,
// 23,900 of 1021 15.3, 14.5 and 20.3, 17,500 of 16384 32, 40 and 54.
constexpr int kPerThread = 2;

// What a launch of assigning writes.
enum { kTokens = 1, kState = 2 };  // table, offsets, positions, slots; lengths, count

__device__ __forceinline__ int held(int64_t x, int64_t most) { return (int)(x < 0 ? 0 : x > most ? most : x); }

// Exclusive prefix sums over the workgroup's threads and their total: a wave's total counts for `most` at most, so that
// 16 of them are a 32-bit number (what is beyond it is not asked for).
// One barrier: s_part is read before the workgroup's next one, and written again behind that.
__device__ __forceinline__ int scan_threads(int a, int *s_part, int &all, int most) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int incl = scan32(a);
    if (lane == 63) s_part[wave] = incl < most ? incl : most;
    __syncthreads();
    const int parts = scan32(lane < kWaves ? s_part[lane & (kWaves - 1)] : 0);
    const int before = __shfl(parts, wave > 0 ? wave - 1 : 0);
    all = lane_value(parts, kWaves - 1);
    return (wave ? before : 0) + incl - a;
}

// The last i with at[i] <= x of kThreads numbers that do not decrease, at[0] <= x.  (Behind the last sequence they are the
// total, which is above every x.)
__device__ __forceinline__ int find_last(const int *at, int x) {
    int lo = 0;
#pragma unroll
    for (int step = kThreads / 2; step > 0; step >>= 1)
        if (at[lo + step] <= x) lo += step;
    return lo;
}

__global__ __launch_bounds__(kThreads) void k_pages_assign(w4a8_pages p, int shift, const int32_t *__restrict__ new_tokens,
                                                           int64_t M, w4a8_batch out, int what) {
    __shared__ int s_part[2][kWaves], s_lack;
    __shared__ int s_token[kThreads], s_page[kThreads], s_old[kThreads];  // from the 1024 sequences' first on
    const int tid = threadIdx.x, rows = (int)M;
    const int64_t P = int64_t(1) << shift, most = p.table_width << shift;
    const int count = held(p.free_count[0], p.num_pages);
    const int64_t share = (int64_t)gridDim.x * kThreads, first = (int64_t)blockIdx.x * kThreads + tid;
    auto taken = [&](int64_t i) {  // the i-th page off the list
        return i < count ? p.free_pages[count - 1 - i] : -1;
    };
    if (tid == 0) s_lack = 0;
    int base = 0, page0 = 0;  // rows and pages in front of the 1024 sequences
    for (int64_t b0 = 0; b0 < p.B; b0 += kThreads) {
        const int64_t b = b0 + tid;
        int old = 0, n = 0;
        if (b < p.B) {
            old = held(p.seq_lens[b], most);
            n = held(new_tokens[b], M);
        }
        // what lies behind row M - 1 is not there: the rows up to a sequence's first are not known before the sum
        int all_tokens, all_pages;
        const int at = scan_threads(n, s_part[0], all_tokens, rows);
        const int row = at < rows - base ? base + at : rows, end = n < rows - row ? row + n : rows;
        all_tokens = all_tokens < rows - base ? all_tokens : rows - base;
        n = end - row;
        const int64_t grown = (int64_t)old + n, len = grown < most ? grown : most;
        const int have = (int)((old + P - 1) >> shift), need = (int)((len + P - 1) >> shift);
        const int lack = (int)((grown + P - 1) >> shift) - need;  // pages that the table has no room for
        if (lack) atomicAdd(&s_lack, lack);
        // (pages, and those that are lacking, are no more than the rows)
        const int page_at = scan_threads(need - have, s_part[1], all_pages, rows);
        s_token[tid] = row - base;
        s_page[tid] = page_at;
        s_old[tid] = old;
        __syncthreads();
        if (what & kTokens) {
            if (blockIdx.x == 0 && b < p.B) {
                out.cu_tokens[b] = row;
                if (b == p.B - 1) out.cu_tokens[p.B] = end;
            }
            for (int64_t i = first; i < all_tokens; i += share) {
                const int q = find_last(s_token, (int)i);
                const int64_t pos = s_old[q] + (i - s_token[q]);
                const int64_t entry = pos >> shift, held_pages = (s_old[q] + P - 1) >> shift;
                int page = -1;
                if (pos < most)
                    page = entry < held_pages ? p.page_table[(b0 + q) * p.table_width + entry]
                                              : taken(page0 + s_page[q] + (entry - held_pages));
                out.positions[base + i] = (int)(pos < INT32_MAX ? pos : INT32_MAX);
                out.slots[base + i] = (uint32_t)page < (uint64_t)p.num_pages ? ((int64_t)page << shift) + (pos & (P - 1)) : -1;
            }
            for (int64_t i = first; i < all_pages; i += share) {
                const int q = find_last(s_page, (int)i);
                const int64_t entry = ((s_old[q] + P - 1) >> shift) + (i - s_page[q]);
                p.page_table[(b0 + q) * p.table_width + entry] = taken(page0 + i);
            }
        }
        if ((what & kState) && blockIdx.x == 0 && b < p.B) out.seq_lens[b] = (int)len;
        base += all_tokens;
        page0 += all_pages;
        __syncthreads();
    }
    if (what & kTokens)
        for (int64_t i = base + first; i < M; i += share) {
            out.positions[i] = 0;
            out.slots[i] = -1;
        }
    if (blockIdx.x == 0 && tid == 0) {
        // (every thread of this workgroup has read the count in front of a barrier)
        if (what & kState) {
            out.free_count[0] = page0 < count ? count - page0 : 0;
            out.missing[0] = (page0 > count ? page0 - count : 0) + s_lack;
        }
    }
}

// From the last sequence to the first, and within one from its last page down.  1024 sequences at a time, or fewer
// where their tables have more than 2^30 entries: page counts are 32-bit numbers then.  What a page costs is the
// instructions of finding it on one compute unit: a thread finds its first one's sequence by bisection among those that
// give pages back, and the next one's by a step.  (All by bisection among all sequences 19.1 us for 23,900 pages, with 64-bit counts 27.)
__global__ __launch_bounds__(kThreads) void k_pages_release(w4a8_pages p, int shift, const int32_t *__restrict__ keep_lens,
                                                            int32_t *lens, int32_t *free_count) {
    __shared__ int s_part[2][kWaves], s_some[kWaves];
    // Of the sequences that give pages back, in turn: pages in front of a sequence's, and its last page's entry in the table and as
    // many more.  Behind the last of them nothing is found.
    __shared__ int s_first[kThreads + 1];
    __shared__ int64_t s_entry[kThreads];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (tid == 0) s_first[kThreads] = INT32_MAX;
    const int P = 1 << shift, most = (int)(p.table_width << shift);
    const int at_once = p.table_width > (int64_t(1) << 20) ? (int)((int64_t(1) << 30) / p.table_width) : kThreads;
    int count = held(p.free_count[0], p.num_pages);
    for (int64_t b0 = 0; b0 < p.B; b0 += at_once) {
        const int seqs = (int)(p.B - b0 < at_once ? p.B - b0 : at_once);
        const int64_t end = p.B - 1 - b0;  // thread 0 has the last one
        int have = 0, gone = 0;
        if (tid < seqs) {
            const int old = held(p.seq_lens[end - tid], most), keep = held(keep_lens[end - tid], old);
            have = (int)(((uint32_t)old + (P - 1)) >> shift);
            gone = have - (int)(((uint32_t)keep + (P - 1)) >> shift);
            lens[end - tid] = keep;
        }
        const uint64_t some = __ballot(gone > 0);
        if (lane == 0) s_some[wave] = __popcll(some);
        int all;
        const int first = scan_threads(gone, s_part[0], all, INT32_MAX);
        const int ranks = scan32(lane < kWaves ? s_some[lane & (kWaves - 1)] : 0), before = __shfl(ranks, wave > 0 ? wave - 1 : 0);
        const int rank = (wave ? before : 0) + __popcll(some & ((uint64_t(1) << lane) - 1));
        if (gone > 0) {
            s_first[rank] = first;
            s_entry[rank] = (end - tid) * p.table_width + have - 1 + first;
        }
        if (tid >= lane_value(ranks, kWaves - 1)) s_first[tid] = INT32_MAX;
        __syncthreads();
        auto load = [&](int i0, int page[kPerThread]) {
            const int i = i0 + tid * kPerThread;
            int q = i < all ? find_last(s_first, i) : 0;
#pragma unroll
            for (int j = 0; j < kPerThread; j++) {
                if (j && i + j < all) q += i + j >= s_first[q + 1];  // (each has a page or more)
                page[j] = i + j < all ? p.page_table[s_entry[q] - (i + j)] : -1;
            }
        };
        int next[kPerThread];
        load(0, next);
        int turn = 1;
        for (int i0 = 0; i0 < all; i0 += kThreads * kPerThread, turn ^= 1) {
            int page[kPerThread];
            int n = 0;
#pragma unroll
            for (int j = 0; j < kPerThread; j++) {
                page[j] = next[j] < p.num_pages ? next[j] : -1;
                n += page[j] >= 0;
            }
            load(i0 + kThreads * kPerThread, next);  // on their way while these are counted
            int taken;
            int at = scan_threads(n, s_part[turn], taken, INT32_MAX);
#pragma unroll
            for (int j = 0; j < kPerThread; j++)
                if (page[j] >= 0) {
                    if (at < p.num_pages - count) p.free_pages[count + at] = page[j];
                    at++;
                }
            count = taken < p.num_pages - count ? count + taken : (int)p.num_pages;
        }
        __syncthreads();
    }
    if (tid == 0) free_count[0] = count;
}

}  // namespace

hipError_t launch_pages_assign(const w4a8_pages &p, int page_shift, const int32_t *new_tokens, int64_t M,
                               const w4a8_batch &out, hipStream_t stream) {
    const bool in_place = out.seq_lens == p.seq_lens || out.free_count == p.free_count;
    int64_t grid = in_place && M <= kAlone ? 1 : (M + kThreads - 1) / kThreads;
    if (grid > 512) grid = 512;
    const bool two = in_place && grid > 1;
    k_pages_assign<<<(unsigned)grid, kThreads, 0, stream>>>(p, page_shift, new_tokens, M, out, two ? kTokens : kTokens | kState);
    if (two) k_pages_assign<<<1, kThreads, 0, stream>>>(p, page_shift, new_tokens, M, out, kState);
    return hipGetLastError();
}

hipError_t launch_pages_release(const w4a8_pages &p, int page_shift, const int32_t *keep, int32_t *lens, int32_t *count,
                                hipStream_t stream) {
    k_pages_release<<<1, kThreads, 0, stream>>>(p, page_shift, keep, lens, count);
    return hipGetLastError();
}

}  // namespace w4a8
