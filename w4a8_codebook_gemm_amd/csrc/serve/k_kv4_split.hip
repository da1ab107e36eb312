// Attention over the paged cache in 4 bits for few query rows a sequence (decode).
//
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp2(s_t - m),  s_t = scale log2(e) q . k_t
//
// HBM bound: 9/16 of a byte a cached value, read once for the few query rows that share its head.
// Rows, products and their layout are the int8 cache's (k_attn_split.hip): the (token, query
// head) pairs of one sequence and one cache head are the columns of v_mfma_f32_16x16x32_f16,
//   S^T [32 positions x 16 rows] = K [positions x D] Q^T,   O^T [D x 16] += V^T P^T,
// with S^T's rows taken as the positions 8 (m / 4) + 4 u + m % 4 of tile u, so that probabilities
// never leave their lane.  Fragments are exact (kv4_tiles.h).  A lane has D / 4 consecutive values of
// a key, so its scale bytes lie together, and D / 16 consecutive values of eight tokens, which are
// one scale group: its eight scale bytes lie together too.  Two tokens' codes are put side by side
// before they become fp16, which is what turns rows of tokens into a fragment.
//
// The unit of a head is a factor of the scores and of the output, so a row's scores need no factor of
// their own and the only statistic is the running maximum m, a whole number: rescaling is exact.
//
// Split: as in the int8 kernel, the tiles of all units form one line that is cut evenly over the
// workgroups; a workgroup's waves take its tiles in turn and join in LDS, and pieces of a cut unit
// through the workspace (join_pieces).
//
// Measured (one token a sequence; a large copy runs at 5.39 TB/s here; the int8 kernel on the same shapes in brackets): 4 x 90k
// to 131k tokens, 24 / 4 heads of 256, 90 to 98 us, 4.8 to 5.2 TB/s (160); 32 x 300 to 16000 60 us, 4.1 (92); 64 x 4000,
// 32 / 8 of 128, 57 us, 5.2 (89), in pages of 16 61 to 66; 256 x 100 to 300 32 us, 1.8 (38); 16 x 8 drafts on 4000 35 us (44),
// on 200 to 4000 31.5 (46), fp32 41 (16 x 8 on 4000); 61 x 5 on 100 to 4000 of 256 75 to 86, fp32 96; 64 x 6 on 100 to 2000 of 128 38, fp32
// 47; 256 x 100 to 300 fp32 35.  Between start and join HBM bounds long calls: their reads alone, the arithmetic taken out, take 91 of
// 101 us (99 where the codes go through the caches).  Drafts are bound by the vector units, which make fragments of the codes.
// 1 x 777 of 256 is 16 us (17), latency: offsets, pages, codes and other workgroups' pieces are reads that wait for each other.
// Tiles have 256 / D parts of 32 positions: two at D 256 take 112 us in place of 102, a whole tile in registers ahead 144 (spills).
#include <type_traits>

#include "kv4_tiles.h"

namespace w4a8 {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
// Workgroups on a compute unit.  1, 2 and 3 with blocks of 16 rows: 64 x 4000 of 128 75, 58 and (spills) 248 us, 1 x 131000 46 and 41.  1
// and 2 with blocks of 32 (2 spills 12 to 31 registers): 64 x 6 drafts on 100 to 2000 47.5 and 37, 200 x 8 on 50 to 500 91 and 74,
// 32 x 16 on 500 to 4000 73 and 66.
constexpr int kPerCu = 2;
// Pieces that join at a node.  2, 8 and 32: 1 x 777 of 256 19.2, 15.9 and 16.2 us, 4 long ones 105, 94 to 98 and 104, 16 x 8
// drafts 44.4, 41.0 and 42.1.
constexpr int kRadix = 8;
// None, 4 and 8 kWaves: 8 x 500 to 1000 of 128 14.1, 11.6 and 11.5 us, 1 x 4000 16.5, 13.0 and 13.4, 16 x 8 drafts on 200 to
// 4000 41.9, 41.0 and 29.7; longer ones take no shares.
constexpr int kMaxShare = 8 * kWaves;
// See Line.  Blocks of 16 rows, kOver 4, 8, 16 and 28: 200 x 100 to 3000 of 128 101.5, 93.8, 95.4 and 101.9 us, 32 ragged of
// 256 59.6, 59.7, 58.1 and 59.9, 4 long ones 104, 98.8, 100.7 and 103.9.  Blocks of 32, 4, 10, 16 and 24: 32 x 16 on 500 to
// 4000 82, 72, 70 and 73, 64 x 6 58, 47.5, 47 and 51, 200 x 8 95, 89, 88 and 90.  kTail 1, 3 and 8: within 2% everywhere.
template <int NB>
constexpr int kOver = NB == 2 ? 10 : 8;
constexpr int kTail = 3;
// Whole units for single waves, which then join nothing: where every wave has one or more, and the longest unit is longer than
// the average by no more tiles than a workgroup has units.  Workgroups' way and waves' (us): 256 x 100 to 300 (32 / 8 of 128) 46 and 32,
// fp32 512 x 300 to 900 136 and 113, 1024 x 100 to 300 (16 / 4 of 64) 83 and 56, 256 x 500 to 2000 99 and 100.5.
constexpr int kSoloOver = 2;  // as kOver (2 and 6: alike)

template <int D, int NB>
struct Layout {
    static constexpr int RB = 16 * NB;
    static constexpr int kSumRows = 4 * kThreads / D;   // rows that join at a time, four values of one a thread
    static constexpr int kItems = RB / kSumRows;
    static constexpr int kRecord = kItems * kThreads * 4 + RB * 4;  // floats of a piece: each thread's values, each row's state
    static constexpr int kRow = D + 4;                  // LDS row, padded
    static constexpr int kLds = kWaves * kSumRows * kRow;  // floats
};

// Bytes that a lane reads of a key's scales and of a value's codes.
template <int N>
struct Bytes;
template <> struct Bytes<1> { typedef uint8_t type; };
template <> struct Bytes<2> { typedef uint16_t type; };
template <> struct Bytes<4> { typedef uint32_t type; };
template <> struct Bytes<8> { typedef uint2 type; };
template <> struct Bytes<16> { typedef uint4 type; };
template <int N>
__device__ __forceinline__ typename Bytes<N>::type load_bytes(const uint8_t *p) {
    return *reinterpret_cast<const typename Bytes<N>::type *>(p);
}
// Codes are read by one lane once: past the caches.
template <int N>
__device__ __forceinline__ typename Bytes<N>::type load_once(const uint8_t *p) {
    if constexpr (N < 4) {
        return __builtin_nontemporal_load(reinterpret_cast<const typename Bytes<N>::type *>(p));
    } else {
        typedef uint32_t type __attribute__((ext_vector_type(N / 4)));
        return __builtin_bit_cast(typename Bytes<N>::type, __builtin_nontemporal_load(reinterpret_cast<const type *>(p)));
    }
}

// kSmall: pages of 16 positions, else of 32 or more: a page for all lanes' part of a tile.  MANY: batches of so many units that
// each wave may have whole ones.
template <int D, int NB, bool BF16, bool kSmall, bool MANY>
__global__ __launch_bounds__(kThreads, kPerCu) void k_kv4_split(Attn4Args a, int wgs) {
    using Lay = Layout<D, NB>;
    constexpr int RB = Lay::RB;
    constexpr int U = 256 / D, T = 32 * U;  // 32-position parts of a tile
    constexpr int kParts = BF16 ? 1 : 2;   // fp16 numbers that make a query value or a probability
    constexpr int kS = D / 32;             // dwords of a key in a lane, steps of the first product
    constexpr int kT = D / 16;             // tiles of O^T
    constexpr int kVB = D / 32;            // bytes of a value row in a lane
    constexpr int kVW = kVB < 4 ? 1 : kVB / 4;  // dwords they are held in
    __shared__ __attribute__((aligned(16))) float s_o[Lay::kLds];
    constexpr int kQ = NB * kParts * kS * 64;  // fragments of a unit's queries
    __shared__ half8_t s_q[(MANY ? kWaves : 1) * kQ];
    __shared__ float s_m[kWaves][RB], s_l[kWaves][RB];
    __shared__ float2 s_all[RB];
    __shared__ int s_flag;
    const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, g = lane >> 4, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    uint32_t *counters = static_cast<uint32_t *>(a.ws);
    float *pieces = reinterpret_cast<float *>(static_cast<char *>(a.ws) + kAttnCounterBytes);

    // the line's length, and this workgroup's part of it: while a part is not more than kMaxShare tiles, units
    // are cut into whole shares of that many tiles, each a workgroup's, if there are workgroups enough
    Work x = seq_work<RB, T>(a, lane);
    auto total = [&](int share, int over, int64_t &units) {
        int64_t sum = 0;
        units = 0;
        for (int64_t b0 = 0; b0 < a.s.B; b0 += 64) {
            if (a.s.B > 64) x = seq_work<RB, T>(a, b0 + lane);
            sum += lane_value(scan64(x.units * on_line(x.tiles, share, over)), 63);
            units += lane_value(scan64(x.units), 63);
        }
        return sum;
    };
    int64_t units, none;
    int64_t line = total(0, 0, units);
    if (line == 0) return;
    bool solo = false;  // uniform over the grid
    if constexpr (MANY) {
        int longest = 0;
        for (int64_t b0 = 0; b0 < a.s.B; b0 += 64) {
            if (a.s.B > 64) x = seq_work<RB, T>(a, b0 + lane);
            longest = longest > x.tiles ? longest : x.tiles;
        }
        solo = units >= (int64_t)wgs * kWaves && max_lanes(longest) - div64(line, units) <= div64(units, wgs);
    }
    auto sync = [&]() {
        if (solo) {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        } else {
            __syncthreads();
        }
    };
    const int step = solo ? 1 : kWaves;
    int share = 0;
    if (!solo) for (int64_t c = div64(line + (int64_t)wgs * kWaves - 1, (int64_t)wgs * kWaves) * kWaves; c <= kMaxShare && share == 0; c += kWaves) {
        const int64_t sum = total((int)c, 0, none);
        if (sum <= (int64_t)wgs * c) {
            share = (int)c;
            line = sum;
        }
    }
    const int over = solo ? kSoloOver : share == 0 && (NB == 1 || units >= wgs) ? kOver<NB> : 0;
    line += over * units;
    const int64_t used = share ? div64(line, share) : solo ? (int64_t)wgs * kWaves : wgs;
    const int64_t w = solo ? (int64_t)blockIdx.x * kWaves + wave : blockIdx.x;
    if (w >= used) return;
    const Line cut{line, used, over, share ? 1 : kTail};
    const int64_t t1 = cut.begin(w + 1);

    int64_t from = 0, from_base = 0, held = -1;  // the 64 sequences that the last unit was in, their place; those in x
    for (int64_t at = cut.begin(w); at < t1;) {
        // the sequence and unit that tile `at` is in
        int64_t base = from_base, b = 0;
        int lo_tile = 0, tiles = 1;
        Seq q{0, 0, 0, 0};
        for (int64_t b0 = from; b0 < a.s.B; b0 += 64) {
            if (a.s.B > 64 && b0 != held) x = seq_work<RB, T>(a, b0 + lane);
            held = b0;
            const int64_t mine = x.units * on_line(x.tiles, share, over), incl = scan64(mine), sum = lane_value(incl, 63);
            if (at < base + sum) {
                const int src = __ffsll((unsigned long long)__ballot(at - base < incl)) - 1;
                from = b0;
                from_base = base;
                b = b0 + src;
                base += lane_value(incl - mine, src);
                lo_tile = lane_value(x.lo, src);
                tiles = lane_value(x.tiles, src);
                q.first = lane_value(x.q.first, src);
                q.n = lane_value(x.q.n, src);
                q.len = lane_value(x.q.len, src);
                q.pos0 = q.len - q.n;
                break;
            }
            base += sum;
        }
        const int length = on_line(tiles, share, over);
        const int64_t unit = div64(at - base, length);
        const int64_t unit0 = base + unit * length;         // the unit's first tile on the line
        const int64_t unit1 = unit0 + length;
        int tile0, tile1;
        if (solo) {  // the units that begin in this wave's part
            tile0 = 0;
            tile1 = tiles;
        }
        if (solo ? unit0 < at : !cut.part(at, t1, unit0, unit1, tiles, tile0, tile1)) {
            at = unit1;
            continue;
        }
        const int rblock = (int)div64(unit, a.c.kv_heads);
        const int h = (int)(unit - (int64_t)rblock * a.c.kv_heads);

        // this lane's rows; a sequence's rows are fewer than 2^31
        const int r0 = rblock * RB;
        const int nrows = q.n * a.group - r0 < RB ? q.n * a.group - r0 : RB;
        int lo[NB], hi[NB];
        float fac[NB];
        auto row_at = [&](int r, int &token, int &head) {  // row r < nrows of the block
            token = (uint32_t)(r0 + r) / (uint32_t)a.group;
            head = h * a.group + (r0 + r - token * a.group);
        };
        // queries, all of a row's values of this lane at once, before the codes are asked for
        RawQ<BF16> raw[NB][kS];
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
            const int r = 16 * nb + n < nrows ? 16 * nb + n : nrows - 1;
            int token, head;
            row_at(r, token, head);
            sees(a, q, token, lo[nb], hi[nb]);
            if (r != 16 * nb + n) hi[nb] = 0;
            const int64_t off = (q.first + token) * a.q_stride + head * D + g * (D / 4);
#pragma unroll
            for (int c = 0; c < kS; c++) raw[nb][c].load(a.q, off + 8 * c);
        }
        // positions that all rows of the block see, and that any does
        int all_lo, all_hi, any_lo, any_hi;
        {
            int t_first, t_last, hd;
            row_at(0, t_first, hd);
            row_at(nrows - 1, t_last, hd);
            sees(a, q, t_first, any_lo, all_hi);
            sees(a, q, t_last, all_lo, any_hi);
        }

        const int end = lo_tile + tile1;
        int first = lo_tile + tile0 + (solo ? 0 : wave);
        if (first < any_lo / T) first += (any_lo / T - first + step - 1) / step * step;
        const int stop = end < tiles_to<T>(any_hi) ? end : tiles_to<T>(any_hi);
        const int P = a.c.page_size, pm = P - 1;
        const int32_t *table = a.s.page_table + b * a.s.table_width;

        // Pages come from 64 entries of the table that the wave's lanes hold: a load of the page itself would be waited for
        // behind the codes that were asked for before it.
        int window0 = 0, window = -1;
        auto find_window = [&](int e) {
            window0 = e;
            // (waited for here, not where it is used on the path that does not come by)
            window = fresh(window0 + lane < a.s.table_width ? table[window0 + lane] : -1);
        };
        auto page_of = [&](int t) {  // page of position t, -1 past the end
            const int e = (t >> a.page_shift) - window0, p = kSmall ? __shfl(window, e) : lane_value(window, e);
            return t < q.len ? p : -1;
        };
        // The slot of position t in a cache of this head's rows; a page that is not there reads page 0, masked.
        auto slot_of = [&](int t, int page, bool &ok) {
            ok = (uint32_t)page < (uint32_t)a.c.num_pages;
            return ((int64_t)(ok ? page : 0) * a.c.kv_heads + h) * P + (t & pm);
        };
        // This lane's places from a part's first position on: in its keys and their scales, its values and theirs.
        const int k_row = 2 * (lane & 12) + (lane & 3);
        const uint32_t k_at = k_row * (D / 2) + g * (D / 8), kc_at = k_row * (D / 16) + g * (D / 64);
        const uint32_t v_at = 8 * g * (D / 2) + n * kVB, vc_at = (uint32_t)(n * (D / 16) / 16) * P + 8 * g;
        // A tile's codes and scale bytes as they lie; `there`: bit x where part x's page of this lane's positions is there.
        struct Codes {
            uint32_t k[U][2][kS], kc[U][2], v[U][8][kVW];
            uint2 vc[U];
            uint32_t there;
        };
        auto load_k = [&](int tile, Codes &c) {
            // (a tile's entries begin with its first position's)
            const int last = (tile * T + (T - 1)) >> a.page_shift;
            if (last - window0 >= 64) find_window((tile * T) >> a.page_shift);
#pragma unroll
            for (int x = 0; x < U; x++) {
                const int t = tile * T + 32 * x, half = kSmall ? 2 * (lane & 8) : 0;  // (small pages: the row's own)
                bool ok;
                const int64_t row = slot_of(t, page_of(t + half), ok);
                const uint8_t *p = a.c.k + row * (D / 2) + (k_at - half * (D / 2)), *sk = a.c.k_scale + row * (D / 16) + (kc_at - half * (D / 16));
#pragma unroll
                for (int u = 0; u < 2; u++) {
                    const uint8_t *pu = p + u * 4 * (D / 2);
                    if constexpr (D >= 128) {
#pragma unroll
                        for (int i = 0; i < kS; i += 4) {
                            const uint4 y = load_once<16>(pu + 4 * i);
                            c.k[x][u][i] = y.x; c.k[x][u][i + 1] = y.y; c.k[x][u][i + 2] = y.z; c.k[x][u][i + 3] = y.w;
                        }
                    } else {
                        const uint2 y = load_once<8>(pu);
                        c.k[x][u][0] = y.x;
                        c.k[x][u][1] = y.y;
                    }
                    c.kc[x][u] = load_bytes<D / 64>(sk + u * 4 * (D / 16));
                }
            }
        };
        auto load_v = [&](int tile, Codes &c) {
            c.there = 0;
#pragma unroll
            for (int x = 0; x < U; x++) {
                const int t = tile * T + 32 * x, half = kSmall ? 8 * (g & 2) : 0;
                bool ok;
                const int64_t row = slot_of(t, page_of(t + half), ok);
                c.there |= (uint32_t)ok << x;
                const uint8_t *p = a.c.v + row * (D / 2) + (v_at - half * (D / 2));
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    if constexpr (kVB == 8) {
                        const uint2 y = load_once<8>(p + j * (D / 2));
                        c.v[x][j][0] = y.x;
                        c.v[x][j][kVW - 1] = y.y;
                    } else {
                        c.v[x][j][0] = load_once<kVB>(p + j * (D / 2));
                    }
                }
                // a block's rows of P scale bytes, one for each group
                const int slot = t & pm;
                c.vc[x] = load_bytes<8>(a.c.v_scale + (row - slot) * (D / 16) + slot + (vc_at - half));
            }
        };
        Codes cd;
        if (first < stop) {  // (a wave without a tile may stand where first * T passes 2^31)
            find_window((first * T) >> a.page_shift);
            load_k(first, cd);
            load_v(first, cd);
        }

        // queries as fp16, into LDS: fragment (block, part, step) as its lanes read it; zeros behind the rows
        int k_exp;
        const float k_part = frexpf(a.c.k_unit[h], &k_exp);
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
            float top = 0.0f;
#pragma unroll
            for (int c = 0; c < kS; c++) {
                float v[8];
                raw[nb][c].values(v);
#pragma unroll
                for (int i = 0; i < 8; i++) top = fmaxf(top, fabsf(v[i]));
            }
            if (16 * nb + n >= nrows) top = 0.0f;
            top = max_xor32(max_xor16(top));
            // the row's largest value at 2^13 .. 2^14: bf16 values are then exact in fp16 down
            // to 2^-28 of it (fp32 as two fp16 numbers to 2^-22 relative), below off by 2^-39
            int ex = 0;
            if (top > 0.0f) frexpf(top, &ex);
            fac[nb] = fmaxf(ldexpf(fabsf(a.scale) * kLog2e * k_part, ex + k_exp - 14 + kValueExp), 0x1p-126f);
            if (solo || wave == nb) {
                half8_t *sq = s_q + (solo ? wave * kQ : 0);
#pragma unroll
                for (int c = 0; c < kS; c++) {
                    half8_t q0, q1;
                    float v[8];
                    raw[nb][c].values(v);
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        const float y = 16 * nb + n < nrows ? ldexpf(a.scale < 0.0f ? -v[i] : v[i], 14 - ex) : 0.0f;
                        q0[i] = (_Float16)y;
                        q1[i] = (_Float16)(y - (float)(_Float16)y);
                    }
                    sq[(nb * kParts * kS + c) * 64 + lane] = q0;
                    if constexpr (kParts == 2) sq[((nb * kParts + 1) * kS + c) * 64 + lane] = q1;
                }
            }
        }
        sync();

        floatx4 o[NB][kT];
        float m[NB], L[NB];
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
            m[nb] = kLow;
            L[nb] = 0.0f;
#pragma unroll
            for (int i = 0; i < kT; i++) o[nb][i] = floatx4{0, 0, 0, 0};
        }
        // a tile's work; kMore: with the next one's loads, without a branch around them, which would have every wait for codes
        // wait for all that is on its way
        auto work = [&](int tile, auto next) {
            constexpr bool kMore = decltype(next)::value;
            floatx4 s[NB][U][2];
#pragma unroll
            for (int nb = 0; nb < NB; nb++)
#pragma unroll
                for (int x = 0; x < U; x++) s[nb][x][0] = s[nb][x][1] = floatx4{0, 0, 0, 0};
            const half8_t *qp = s_q + (solo ? wave * kQ : 0) + fresh(lane);
            half8_t qf[2][NB][kParts];  // this step's and the next one's
            auto take_q = [&](int c) {
#pragma unroll
                for (int nb = 0; nb < NB; nb++)
#pragma unroll
                    for (int pt = 0; pt < kParts; pt++) qf[c & 1][nb][pt] = qp[((nb * kParts + pt) * kS + c) * 64];
            };
            take_q(0);
#pragma unroll
            for (int c = 0; c < kS; c++) {
                if (c + 1 < kS) take_q(c + 1);
#pragma unroll
                for (int x = 0; x < U; x++)
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        // 16 values a scale: two dwords
                        const uint32_t b = cd.kc[x][u];
                        const half2_t sc = c < 2 ? scale_both<0>(b) : c < 4 ? scale_both<1>(b) : c < 6 ? scale_both<2>(b) : scale_both<3>(b);
                        const half8_t k = values_natural(cd.k[x][u][c], sc);
#pragma unroll
                        for (int nb = 0; nb < NB; nb++)
#pragma unroll
                            for (int pt = 0; pt < kParts; pt++)
                                s[nb][x][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, qf[c & 1][nb][pt], s[nb][x][u], 0, 0, 0);
                    }
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (kMore) load_k(tile + step, cd);
            __builtin_amdgcn_sched_barrier(0);
            const uint32_t there = cd.there;
            const bool whole = tile * T >= all_lo && all_hi - tile * T >= T && __all(there == (1u << U) - 1);
            half8_t pf[NB][U][kParts];
#pragma unroll
            for (int nb = 0; nb < NB; nb++) {
                if (!whole) {
#pragma unroll
                    for (int y = 0; y < U; y++) {
                        const int t = tile * T + 32 * y + 8 * g;
                        const bool ok = there >> y & 1;
#pragma unroll
                        for (int j = 0; j < 8; j++) {
                            const bool see = ok & (t + j >= lo[nb]) & (t + j < hi[nb]);
                            s[nb][y][j >> 2][j & 3] = see ? s[nb][y][j >> 2][j & 3] : -INFINITY;
                        }
                    }
                }
                float all = -INFINITY;
#pragma unroll
                for (int y = 0; y < U; y++)
#pragma unroll
                    for (int j = 0; j < 8; j++) all = fmaxf(all, s[nb][y][j >> 2][j & 3]);
                all = max_xor32(max_xor16(all));
                const float mn = running_maximum(m[nb], all * fac[nb]);
                const float down = m[nb] - mn;             // <= 0
                const float c = (float)kProbExp - mn;
                float sum = 0.0f;
#pragma unroll
                for (int y = 0; y < U; y++) {
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const float p = __builtin_amdgcn_exp2f(fmaf(s[nb][y][j >> 2][j & 3], fac[nb], c));  // 2^14 at most
                        sum += p;
                        const _Float16 p0 = (_Float16)p;
                        pf[nb][y][0][j] = p0;
                        if constexpr (kParts == 2) pf[nb][y][1][j] = (_Float16)(p - (float)p0);
                    }
                }
                const float turn = pow2_down(down);
                L[nb] = L[nb] * turn + sum;
                if (__any(down < 0.0f)) {
#pragma unroll
                    for (int i = 0; i < kT; i++) o[nb][i] *= turn;
                }
                m[nb] = mn;
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int y = 0; y < U; y++) {
                const half2_t sv[4] = {scale_pair<0>(cd.vc[y].x), scale_pair<2>(cd.vc[y].x), scale_pair<0>(cd.vc[y].y), scale_pair<2>(cd.vc[y].y)};
#pragma unroll
                for (int i = 0; i < kVW; i++)
#pragma unroll
                    for (int odd = 0; odd < 2; odd++) {
                        uint32_t d[4];
#pragma unroll
                        for (int j = 0; j < 4; j++)
                            d[j] = odd ? odd_codes(cd.v[y][2 * j][i], cd.v[y][2 * j + 1][i]) : even_codes(cd.v[y][2 * j][i], cd.v[y][2 * j + 1][i]);
                        auto tile_of = [&](auto byte) {
                            constexpr int J = decltype(byte)::value;
                            const half8_t f = __builtin_bit_cast(half8_t, make_uint4(codes_times<J>(d[0], sv[0]), codes_times<J>(d[1], sv[1]),
                                                                                     codes_times<J>(d[2], sv[2]), codes_times<J>(d[3], sv[3])));
                            const int k = 8 * i + 2 * J + odd;
#pragma unroll
                            for (int nb = 0; nb < NB; nb++)
#pragma unroll
                                for (int pt = 0; pt < kParts; pt++)
                                    o[nb][k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, pf[nb][y][pt], o[nb][k], 0, 0, 0);
                        };
                        tile_of(std::integral_constant<int, 0>());
                        tile_of(std::integral_constant<int, 1>());
                        if constexpr (kVB >= 4) {
                            tile_of(std::integral_constant<int, 2>());
                            tile_of(std::integral_constant<int, 3>());
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
            }
            if constexpr (kMore) load_v(tile + step, cd);
        };
        if (first < stop) {
            int tile = first;
            for (; tile + step < stop; tile += step) work(tile, std::true_type());
            work(tile, std::false_type());
        }

        // join the waves: the column's sum first (a lane has summed its own positions)
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
            L[nb] += __shfl_xor(L[nb], 16);
            L[nb] += __shfl_xor(L[nb], 32);
            if (g == 0) {
                s_m[wave][16 * nb + n] = m[nb];
                s_l[wave][16 * nb + n] = L[nb];
            }
        }
        // a wave's rows x kSumRows .. into LDS, in order of their values
        constexpr int kItems = Lay::kItems, kSumRows = Lay::kSumRows;
        auto spread = [&](int x) {
#pragma unroll
            for (int nb = 0; nb < NB; nb++) {
                const int r = 16 * nb + n - x * kSumRows;
                if (r >= 0 && r < kSumRows) {
                    float *p = s_o + (wave * kSumRows + r) * Lay::kRow;
#pragma unroll
                    for (int ii = 0; ii < 4; ii++)
#pragma unroll
                        for (int i = 0; i < kT; i += 4)
                            *reinterpret_cast<float4 *>(p + (4 * g + ii) * kT + i) =
                                make_float4(o[nb][i][ii], o[nb][i + 1][ii], o[nb][i + 2][ii], o[nb][i + 3][ii]);
                }
            }
        };
        int v_exp;
        const float v_part = frexpf(a.c.v_unit[h], &v_exp);
        // four values of row r, from value d on, to o; the sum of the probabilities carries the same 2^14 as the products
        auto finish = [&](int r, int d, const float v[4], float L) {
            const float inv = L > 0.0f ? v_part / L : 0.0f;
            float y[4];
#pragma unroll
            for (int i = 0; i < 4; i++) y[i] = ldexpf(v[i] * inv, v_exp + kValueExp);
            int token, head;
            row_at(r, token, head);
            const int64_t off = ((q.first + token) * a.hq + head) * D + d;
            if constexpr (BF16)
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.o) + off) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
            else
                *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + off) = make_float4(y[0], y[1], y[2], y[3]);
        };
        sync();
        if (solo) {
#pragma unroll
            for (int x = 0; x < kItems; x++) {
                if (x * kSumRows >= nrows) break;
                spread(x);
                sync();
#pragma unroll
                for (int y = 0; y < kSumRows * D / 256; y++) {
                    const int i = 64 * y + lane, sr = i / (D / 4), sd = 4 * (i % (D / 4)), r = x * kSumRows + sr;
                    const float4 f = *reinterpret_cast<const float4 *>(s_o + (wave * kSumRows + sr) * Lay::kRow + sd);
                    const float v[4] = {f.x, f.y, f.z, f.w};
                    if (r < nrows) finish(r, sd, v, s_l[wave][r]);
                }
                sync();
            }
            at = unit1;
            continue;
        }
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
            const int r = 16 * nb + n;
            float mm = s_m[0][r];
            for (int x = 1; x < kWaves; x++) mm = fmaxf(mm, s_m[x][r]);
            if (wave == nb && g == 0) {
                float l = 0.0f;
                for (int x = 0; x < kWaves; x++) l += s_l[x][r] * pow2_down(s_m[x][r] - mm);
                s_all[r] = make_float2(mm, l);
            }
            const float y = pow2_down(m[nb] - mm);
#pragma unroll
            for (int i = 0; i < kT; i++) o[nb][i] *= y;
        }
        // sum over the waves, kSumRows rows at a time; a thread ends with four values of a row of each
        const int ir = tid / (D / 4), id = 4 * (tid % (D / 4));
        float v[kItems][4];
        State st[kItems];
#pragma unroll
        for (int x = 0; x < kItems; x++) {
            const int q0 = x * kSumRows;
            if (q0 >= nrows) break;
            spread(x);
            __syncthreads();
            v[x][0] = v[x][1] = v[x][2] = v[x][3] = 0.0f;
            {
#pragma unroll
                for (int y = 0; y < kWaves; y++) {
                    const float4 f = *reinterpret_cast<const float4 *>(s_o + (y * kSumRows + ir) * Lay::kRow + id);
                    v[x][0] += f.x; v[x][1] += f.y; v[x][2] += f.z; v[x][3] += f.w;
                }
                const float2 f = s_all[q0 + ir];
                st[x] = State{f.x, 0.0f, f.y};
            }
            __syncthreads();
        }
        bool write = true;
        if (tile1 - tile0 < tiles) {
            const int64_t w_first = cut.first(unit0), w_end = cut.last(unit1);
            auto slot = [&](unsigned x) { return shared_piece(pieces + (2 * (w_first + x) + (x == 0 ? 1 : 0)) * Lay::kRecord, 4 * Lay::kRecord); };
            write = join_pieces<kRadix>(counters, w_first, w, w_end, &s_flag, [&](unsigned y) {
                const __amdgpu_buffer_rsrc_t p = slot(y);
#pragma unroll
                for (int x = 0; x < kItems; x++) {
                    const int r = x * kSumRows + ir;
                    if (r < nrows) {
                        put_shared4(p, (x * kThreads + tid) * 16, v[x][0], v[x][1], v[x][2], v[x][3]);
                        if (id == 0) put_shared4(p, (kItems * kThreads + r) * 16, st[x].m, st[x].E, st[x].L, 0.0f);
                    }
                }
            }, [&](unsigned y0, unsigned step, unsigned pieces_here) {
#pragma unroll
                for (int x = 0; x < kItems; x++) {
                    const int r = x * kSumRows + ir;
                    if (r >= nrows) break;
                    st[x] = State{kLow, 0.0f, 0.0f};
                    v[x][0] = v[x][1] = v[x][2] = v[x][3] = 0.0f;
                    auto some = [&](auto count, unsigned y) {  // so many slots from y on, their loads together
                        constexpr int kCount = decltype(count)::value;
                        floatx4 f[kCount], t[kCount];
#pragma unroll
                        for (int z = 0; z < kCount; z++) {
                            const __amdgpu_buffer_rsrc_t p = slot(y0 + (y + z) * step);
                            f[z] = get_shared4(p, (x * kThreads + tid) * 16);
                            t[z] = get_shared4(p, (kItems * kThreads + r) * 16);
                        }
#pragma unroll
                        for (int z = 0; z < kCount; z++) {
                            float qa, qb;
                            st[x] = join(st[x], State{t[z][0], t[z][1], t[z][2]}, qa, qb);
#pragma unroll
                            for (int i = 0; i < 4; i++) v[x][i] = v[x][i] * qa + f[z][i] * qb;
                        }
                    };
                    unsigned y = 0;
                    for (; y + 4 <= pieces_here; y += 4) some(std::integral_constant<int, 4>(), y);
                    for (; y < pieces_here; y++) some(std::integral_constant<int, 1>(), y);
                }
            });
        }
        if (write) {
#pragma unroll
            for (int x = 0; x < kItems; x++) {
                const int r = x * kSumRows + ir;
                if (r < nrows) finish(r, id, v[x], st[x].L);
            }
        }
        at = unit1;
    }
}

template <int D, int NB>
hipError_t launch_nb(const Attn4Args &a, int bf16, int num_cu, hipStream_t stream) {
    const int wgs = kPerCu * num_cu;
    auto pick = [&](auto many) {
        constexpr bool M = decltype(many)::value;
        return a.page_shift == 4 ? (bf16 ? k_kv4_split<D, NB, true, true, M> : k_kv4_split<D, NB, false, true, M>)
                                 : (bf16 ? k_kv4_split<D, NB, true, false, M> : k_kv4_split<D, NB, false, false, M>);
    };
    auto f = pick(std::false_type());
    // (at head_dim 256 the registers do not hold what both ways need)
    if constexpr (NB == 1 && D < 256) {
        if (a.s.B * a.c.kv_heads >= (int64_t)wgs * kWaves) f = pick(std::true_type());
    }
    f<<<wgs, kThreads, 0, stream>>>(a, wgs);
    return hipGetLastError();
}

template <int D>
int64_t bytes_d(int num_cu) {
    return 4 * 2 * (int64_t)kPerCu * num_cu * Layout<D, D < 256 ? 2 : 1>::kRecord;
}

}  // namespace

int64_t kv4_split_bytes(int head_dim, int num_cu) {
    return head_dim == 64 ? bytes_d<64>(num_cu) : head_dim == 128 ? bytes_d<128>(num_cu) : bytes_d<256>(num_cu);
}

// Blocks of 16 rows read a sequence's codes once for each, at twice the work in flight; blocks of 32 pay where units are many.
// Blocks of 16 and 32 (us).  24 to 32 rows, 32 / 8 heads of 128: 16 x 6 on 4000 35.0 and 32.9, 16 x 8 37.3 and 35.3, 64 x 6 on
// 100 to 2000 49 and 37; fewer sequences and heads, 30 x 8 on 2000 to 9000 (8 / 2 of 128) 31.9 and 39.0, 16 x 8 (16 / 4 of 64)
// 22.9 and 28.3.  33 to 64 rows: 32 x 16 on 500 to 4000 79 and 64, 8 x 16 on 10k to 20k 107 and 85, 4 x 16 on 30k to 60k 145
// and 116; 8 x 16 on 1000 to 4000 29.9 and 31.0, 2 x 12 on 1000 to 9000 25.7 and 36.5.  At head_dim 256 blocks of 32 leave one
// wave a SIMD: 61 x 5 on 100 to 4000 74 and 120, 4 x 8 on 30k to 60k 121 and 138, 8 x 10 on 4000 38 and 42.
hipError_t launch_kv4_split(const Attn4Args &a, int bf16, int64_t rows, int num_cu, hipStream_t stream) {
    const int64_t heads = a.s.B * a.c.kv_heads;
    const bool wide = rows > 16 && heads >= (rows > 32 ? num_cu / 8 : num_cu / 2);
    switch (a.c.head_dim) {
        case 64: return wide ? launch_nb<64, 2>(a, bf16, num_cu, stream) : launch_nb<64, 1>(a, bf16, num_cu, stream);
        case 128: return wide ? launch_nb<128, 2>(a, bf16, num_cu, stream) : launch_nb<128, 1>(a, bf16, num_cu, stream);
        default: return launch_nb<256, 1>(a, bf16, num_cu, stream);
    }
}

}  // namespace w4a8
