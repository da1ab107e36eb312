// Attention over the int8 paged cache for few query rows a sequence (decode).
//
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp2(s_t - m),  s_t = scale log2(e) q . k_t
//
// HBM bound: each code is read once and used for the few query rows that share its head.
// The rows of a unit are the (token, query head) pairs of one sequence and one cache head, in
// blocks of 16 NB; they are the columns of v_mfma_f32_16x16x32_f16:
//   S^T [32 positions x 16 rows] = K [positions x D] Q^T,   O^T [D x 16] += V^T P^T.
// With S^T's rows taken as the positions 8 (m / 4) + 4 u + m % 4 of tile u, a lane's eight
// scores are those of eight consecutive positions of its row, which is the fragment the
// second product wants: probabilities never leave their lane.  Codes become fp16 in
// registers: K rows by bytes in order, V by a permute that transposes 2 tokens x 1 value, one permute and
// one packed addition (keys) or multiply-add (values) for two codes.  A wave takes 8192 / D positions at a time, the
// next ones' codes (16 KiB) on their way while it works; queries lie in LDS, shared by the waves.
//
// The running maximum m and the exponent E are whole numbers: with e the exponent of a page's
// value scale sv < 2^e, a probability enters the second product as p sv 2^(14 - E), E the
// largest (m_page - m) + e so far, so it is below 2^14 whatever the pages' scales, and every
// rescaling is by a power of two, exact.  o = O 2^(9 - 14 + E) / sum p (codes are 2^9 less).
//
// Split: the tiles of all units form one line that is cut evenly over the workgroups whatever the
// lengths are; a workgroup's waves take its tiles in turn and join in LDS.  The pieces of a unit
// that is cut are joined through the workspace (join_pieces).  Where units are many and alike, waves have whole ones instead.
//
// Measured (24 / 4 heads of 256, one token a sequence): 4 x 90k to 131k tokens 170 to 175 us, 5.6 TB/s of 6.0 that a
// plain read reaches here; 32 x 300 to 16000 103 to 107 us, 5.0 TB/s; 64 x 4000 (32 / 8 of 128) 95 us, 5.5 TB/s; fp32
// 4 x 30k to 60k 85 us, 4.6 TB/s; blocks of 32 rows, 16 x 8 tokens on 4000 (32 / 8 of 128), 42 us, 3.1 TB/s.
// Probabilities as two fp16 numbers for bf16 rows too are 2% slower on long contexts and 4 to 8% with more rows
// (183 and 187 us, 43.8 and 47.0), for outputs that bf16 rounds to 2^-9.  At head_dim 256 the kernels spill
// 8 to 17 registers, none of them in the loop over tiles: each unit pays for it once.
// Between a workgroup's first tile and its join it streams at 6.3 TB/s; what is lost is starting and joining, some 12 us
// a call: 1 x 777 tokens is 16.3 us, of them 1.6 the line, 1.4 finding the unit, 3.9 rows, pages and queries (each
// waits for a read), 1.7 the tiles, 1.8 the waves' join and 2.2 the workgroups'.
#include <type_traits>

#include "attn_tiles.h"

namespace w4a8 {
namespace {

constexpr int kWaves = 4;         // two workgroups on a compute unit: one streams while the other joins
constexpr int kThreads = 64 * kWaves;

// Values are read by one lane once: past the caches.
template <class V>
__device__ __forceinline__ V load_once(const int8_t *p) {
    typedef uint32_t type __attribute__((ext_vector_type(sizeof(V) / 4)));
    return __builtin_bit_cast(V, __builtin_nontemporal_load(reinterpret_cast<const type *>(p)));
}

template <int D>
struct VLoad;
template <> struct VLoad<256> { typedef uint4 type; };
template <> struct VLoad<128> { typedef uint2 type; };
template <> struct VLoad<64> { typedef uint32_t type; };

// Workgroups on a compute unit: blocks of 32 rows need the registers of two.
template <int NB>
constexpr int kPerCu = NB == 2 ? 1 : 2;
constexpr int kRadix = 8;        // pieces that join at a node

// Measured (us; 0, 16 and 32 tiles): 8 x 500 to 1000 tokens (32 / 8 heads of 128) 17.5, 14.5 and 14.4; 1 x 777 of 24 / 4 of
// 256 20.6, 18.9 and 18.9; 16 x 8 tokens on 200 to 4000 49.1, 49.1 and 41.6; longer ones take no shares.
constexpr int kMaxShare = 4 * kWaves;
// See Line: a unit's start and end cost some 8 us, a workgroup's tile 1 (blocks of 16 rows) or 2.  kOver at 2, as it is, and at
// 16: 32 ragged sequences 115, 113 and 111 us, 100 x 100 to 3000 tokens (32 / 8 of 128) 83, 77.5 and 80, 4 long ones 186, 183 and
// 182; blocks of 32 rows, 32 x 16 tokens on 500 to 4000, 115, 106 and 93.  kTail at 1, 3 and 8: 112.5, 112.9 and 112.3 for the
// ragged ones, 52, 49 and 49 for 16 x 8 tokens, 108, 106 and 104 for 32 x 16.
template <int NB>
constexpr int kOver = NB == 2 ? 4 : 8;
constexpr int kTail = 3;
// Whole units for single waves, which then join nothing: where every wave has one or more, and the longest unit is longer than
// the average by no more tiles than a workgroup has units.  (A wave that is left with the longest takes some 1.5 us a tile; a
// workgroup starts and joins its units one after the other.)  32 / 8 heads of 128, workgroups' way and waves': 256 x 100 to 300
// tokens 54 and 40 us, 256 x 500 to 2000 143 and 154, 512 of them 259 and 272, 1024 510 and 510, 256 x 2000 194 and
// 185, fp32 512 x 300 to 900 178 and 155.  kSoloOver: as kOver.
constexpr int kSoloOver = 2;

template <int D, int NB>
struct Layout {
    static constexpr int RB = 16 * NB;
    static constexpr int kSumRows = 4 * kThreads / D;   // rows that join at a time, four values of one a thread
    static constexpr int kItems = RB / kSumRows;
    static constexpr int kRecord = kItems * kThreads * 4 + RB * 4;  // floats of a piece: each thread's values, each row's state
    static constexpr int kRow = D + 4;                  // LDS row, padded
    static constexpr int kLds = kWaves * kSumRows * kRow;  // floats
};

// MANY: batches of so many units that each wave may have whole ones.
template <int D, int NB, bool BF16, bool MANY>
__global__ __launch_bounds__(kThreads, kPerCu<NB>) void k_attn_split(AttnArgs a, int wgs) {
    using Lay = Layout<D, NB>;
    using VT = typename VLoad<D>::type;
    constexpr int RB = Lay::RB;
    constexpr int U = 256 / D, T = 32 * U;  // 32-position parts of a tile
    constexpr int kParts = BF16 ? 1 : 2;   // fp16 numbers that make a query value or a probability
    constexpr int kC = D / 64;             // 16-byte chunks of a key row, dwords of a value row in a lane
    constexpr int kT = D / 16;             // tiles of O^T
    __shared__ __attribute__((aligned(16))) float s_o[Lay::kLds];
    constexpr int kQ = NB * kParts * 2 * kC * 64;  // fragments of a unit's queries
    __shared__ half8_t s_q[(MANY ? kWaves : 1) * kQ];
    __shared__ float s_m[kWaves][RB], s_e[kWaves][RB], s_l[kWaves][RB];
    __shared__ float4 s_all[RB];
    __shared__ int s_flag;
    const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, g = lane >> 4;
    const int wave = MANY ? __builtin_amdgcn_readfirstlane(tid >> 6) : tid >> 6;
    uint32_t *counters = static_cast<uint32_t *>(a.ws);
    float *pieces = reinterpret_cast<float *>(static_cast<char *>(a.ws) + kAttnCounterBytes);

    // the line's length, and this workgroup's part of it
    // Even parts may end inside a unit, and a workgroup that has parts of two pays twice for starting
    // and joining.  While a part is not more than kMaxShare tiles, units are cut into whole shares of
    // that many tiles instead, each a workgroup's, if there are workgroups enough.
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
#pragma unroll
        for (int i = 1; i < 64; i <<= 1) {
            const int o = __shfl_xor(longest, i);
            longest = longest > o ? longest : o;
        }
        solo = units >= (int64_t)wgs * kWaves && __builtin_amdgcn_readfirstlane(longest) - div64(line, units) <= div64(units, wgs);
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
    // with fewer units than workgroups nearly every part is one piece and pays the same: blocks of 32 rows are
    // then better cut evenly (16 x 8 tokens on 4k 46 us, 49 with kOver); blocks of 16 are not (32 ragged
    // sequences 114 us evenly, 112 with kOver, 4 long ones 184 and 181)
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
        RawQ<BF16> raw[NB][2 * kC];
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
            const int r = 16 * nb + n < nrows ? 16 * nb + n : nrows - 1;
            int token, head;
            row_at(r, token, head);
            sees(a, q, token, lo[nb], hi[nb]);
            if (r != 16 * nb + n) hi[nb] = 0;
            const int64_t off = (q.first + token) * a.q_stride + head * D + 16 * g;
#pragma unroll
            for (int c = 0; c < kC; c++)
#pragma unroll
                for (int u = 0; u < 2; u++) raw[nb][2 * c + u].load(a.q, off + 64 * c + 8 * u);
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
        const bool small = a.page_shift == 4;  // two pages in 32 positions
        const int32_t *table = a.s.page_table + b * a.s.table_width;

        auto page_of = [&](int t) {  // page of position t, -1 past the end
            return t < q.len ? table[t >> a.page_shift] : -1;
        };
        auto block_of = [&](int page) {  // its block of this head; a page that is not there reads page 0, masked
            return (int64_t)((uint32_t)page < (uint32_t)a.c.num_pages ? page : 0) * a.c.kv_heads + h;
        };
        uint4 kr[U][2][kC];
        VT vr[U][8];
        float ks[U], vs[U];
        int pk[U], ps[U];       // pages of the tile to load next, of this lane's key row and of its positions
        auto find_pages = [&](int tile) {
            const int l = fresh(lane);
#pragma unroll
            for (int x = 0; x < U; x++) {
                const int t = tile * T + 32 * x;
                pk[x] = page_of(t + (small ? 2 * (l & 8) : 0));
                ps[x] = page_of(t + (small ? (l & 32) >> 1 : 0));
            }
        };
        auto load_k = [&](int tile) {
            const int l = fresh(lane);
#pragma unroll
            for (int x = 0; x < U; x++) {
                const int8_t *p = a.c.k + (block_of(pk[x]) * P + ((tile * T + 32 * x + 2 * (l & 12) + (l & 3)) & pm)) * D + (l >> 4) * 16;
#pragma unroll
                for (int u = 0; u < 2; u++)
#pragma unroll
                    for (int c = 0; c < kC; c++) kr[x][u][c] = *reinterpret_cast<const uint4 *>(p + 4 * u * D + 64 * c);
            }
        };
        auto load_v = [&](int tile) {
            const int l = fresh(lane);
#pragma unroll
            for (int x = 0; x < U; x++) {
                const int8_t *p = a.c.v + (block_of(ps[x]) * P + ((tile * T + 32 * x + (l >> 4) * 8) & pm)) * D + (l & 15) * (D / 16);
#pragma unroll
                for (int j = 0; j < 8; j++) vr[x][j] = load_once<VT>(p + j * D);
            }
        };
        // value scale -1 where the page is not there
        auto load_scales = [&]() {
#pragma unroll
            for (int x = 0; x < U; x++) {
                const int64_t blk = block_of(ps[x]);
                ks[x] = a.c.k_scale[blk];
                vs[x] = (uint32_t)ps[x] < (uint32_t)a.c.num_pages ? a.c.v_scale[blk] : -1.0f;
            }
        };
        if (first < stop) {
            find_pages(first);
            load_scales();
            load_k(first);
            load_v(first);
            if (first + step < stop) find_pages(first + step);
        }

        // queries as fp16, into LDS: fragment (block, part, step) as its lanes read it; zeros behind the rows
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
            float top = 0.0f;
#pragma unroll
            for (int c = 0; c < 2 * kC; c++) {
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
            fac[nb] = ldexpf(fabsf(a.scale) * kLog2e, ex - 14);
            if (solo || wave == nb) {
                half8_t *sq = s_q + (solo ? wave * kQ : 0);
#pragma unroll
                for (int c = 0; c < 2 * kC; c++) {
                    half8_t q0, q1;
                    float v[8];
                    raw[nb][c].values(v);
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        const float x = 16 * nb + n < nrows ? ldexpf(a.scale < 0.0f ? -v[i] : v[i], 14 - ex) : 0.0f;
                        q0[i] = (_Float16)x;
                        q1[i] = (_Float16)(x - (float)(_Float16)x);
                    }
                    sq[(nb * kParts * 2 * kC + c) * 64 + lane] = q0;
                    if constexpr (kParts == 2) sq[((nb * kParts + 1) * 2 * kC + c) * 64 + lane] = q1;
                }
            }
        }
        sync();

        floatx4 o[NB][kT];
        float m[NB], E[NB], L[NB];
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
            m[nb] = kLow;
            E[nb] = 0.0f;
            L[nb] = 0.0f;
#pragma unroll
            for (int i = 0; i < kT; i++) o[nb][i] = floatx4{0, 0, 0, 0};
        }
        for (int tile = first; tile < stop; tile += step) {
            const bool more = tile + step < stop;
            floatx4 s[NB][U][2];
#pragma unroll
            for (int nb = 0; nb < NB; nb++)
#pragma unroll
                for (int x = 0; x < U; x++) s[nb][x][0] = s[nb][x][1] = floatx4{0, 0, 0, 0};
            const half8_t *qp = s_q + (solo ? wave * kQ : 0) + fresh(lane);
#pragma unroll
            for (int c = 0; c < kC; c++) {
                half8_t qf[NB][kParts][2];
#pragma unroll
                for (int nb = 0; nb < NB; nb++)
#pragma unroll
                    for (int pt = 0; pt < kParts; pt++)
#pragma unroll
                        for (int i = 0; i < 2; i++) qf[nb][pt][i] = qp[((nb * kParts + pt) * 2 * kC + 2 * c + i) * 64];
#pragma unroll
                for (int x = 0; x < U; x++)
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        const half8_t k0 = codes_natural(kr[x][u][c].x, kr[x][u][c].y), k1 = codes_natural(kr[x][u][c].z, kr[x][u][c].w);
#pragma unroll
                        for (int nb = 0; nb < NB; nb++)
#pragma unroll
                            for (int pt = 0; pt < kParts; pt++) {
                                s[nb][x][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, qf[nb][pt][0], s[nb][x][u], 0, 0, 0);
                                s[nb][x][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, qf[nb][pt][1], s[nb][x][u], 0, 0, 0);
                            }
                    }
            }
            float tks[U], tvs[U];
#pragma unroll
            for (int x = 0; x < U; x++) {
                tks[x] = ks[x];
                tvs[x] = vs[x];
            }
            if (more) {
                load_scales();
                load_k(tile + step);
            }
            bool whole = tile * T >= all_lo && all_hi - tile * T >= T;
#pragma unroll
            for (int x = 0; x < U; x++) whole = whole && __all(tvs[x] >= 0.0f);
            half8_t pf[NB][U][kParts];
#pragma unroll
            for (int nb = 0; nb < NB; nb++) {
                float x[U][8], mx[U], all = -INFINITY;
                int e[U];
#pragma unroll
                for (int y = 0; y < U; y++) {
                    const float f = fac[nb] * tks[y];
                    mx[y] = -INFINITY;
#pragma unroll
                    for (int j = 0; j < 8; j++) x[y][j] = s[nb][y][j >> 2][j & 3] * f;
                    if (!whole) {
                        const int t = tile * T + 32 * y + 8 * g;
#pragma unroll
                        for (int j = 0; j < 8; j++) {
                            const bool see = (tvs[y] >= 0.0f) & (t + j >= lo[nb]) & (t + j < hi[nb]);
                            x[y][j] = see ? x[y][j] : -INFINITY;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 8; j++) mx[y] = fmaxf(mx[y], x[y][j]);
                    all = fmaxf(all, mx[y]);
                }
                all = max_xor32(max_xor16(all));
                const float mn = fmaxf(m[nb], ceilf(all));
                const float down = m[nb] - mn;             // <= 0
                // the pages this lane's positions are in; of a page that is not seen the scale, whatever it
                // holds, stays out
                float top = -INFINITY;
#pragma unroll
                for (int y = 0; y < U; y++) {
                    e[y] = kZeroExp;
                    if (mx[y] > -INFINITY && tvs[y] > 0.0f) frexpf(tvs[y], &e[y]);
                    top = fmaxf(top, (ceilf(mx[y]) - mn) + (float)e[y]);
                }
                top = max_xor32(max_xor16(top));
                // With bf16 blocks of 32 rows E grows by 4 more than it has to, so that it seldom does (8 x 10 tokens on
                // 4000, 24 / 4 heads of 256, 54.8 us, 56.4 by no more; 8 x 16 of 128 43.5 and 44.2).  That takes 4 bits off
                // weights below fp16's normal range.  Blocks of 16 rows take the same time either way, fp32 wants the bits.
                const float En = top > E[nb] + down ? top + (BF16 && NB == 2 ? 4.0f : 0.0f) : E[nb] + down;
                const float turn = down + (E[nb] - En);    // exponent of the rescaling of o, <= 0
                float sum = 0.0f;
#pragma unroll
                for (int y = 0; y < U; y++) {
                    const float w = e[y] > kZeroExp ? fminf(ldexpf(tvs[y], (int)((float)kProbExp - En)), 1e38f) : 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const float p = __builtin_amdgcn_exp2f(x[y][j] - mn);
                        sum += p;
                        const float v = fminf(p * w, 32768.0f);
                        const _Float16 p0 = (_Float16)v;
                        pf[nb][y][0][j] = p0;
                        if constexpr (kParts == 2) pf[nb][y][1][j] = (_Float16)(v - (float)p0);
                    }
                }
                L[nb] = L[nb] * pow2_down(down) + sum;
                if (__any(turn < 0.0f)) {
                    const float q = pow2_down(turn);
#pragma unroll
                    for (int i = 0; i < kT; i++) o[nb][i] *= q;
                }
                m[nb] = mn;
                E[nb] = En;
            }
#pragma unroll
            for (int x = 0; x < U; x++) {
                auto dword = [&](int j, int i) -> uint32_t {
                    if constexpr (D == 256) return (i == 0 ? vr[x][j].x : i == 1 ? vr[x][j].y : i == 2 ? vr[x][j].z : vr[x][j].w) ^ kSign4;
                    else if constexpr (D == 128) return (i == 0 ? vr[x][j].x : vr[x][j].y) ^ kSign4;
                    else return vr[x][j] ^ kSign4;
                };
#pragma unroll
                for (int i = 0; i < kC; i++) {
                    uint32_t d[8];
#pragma unroll
                    for (int j = 0; j < 8; j++) d[j] = dword(j, i);
                    half8_t f[4];
                    f[0] = __builtin_bit_cast(half8_t, make_uint4(codes_pair<0>(d[0], d[1]), codes_pair<0>(d[2], d[3]), codes_pair<0>(d[4], d[5]), codes_pair<0>(d[6], d[7])));
                    f[1] = __builtin_bit_cast(half8_t, make_uint4(codes_pair<1>(d[0], d[1]), codes_pair<1>(d[2], d[3]), codes_pair<1>(d[4], d[5]), codes_pair<1>(d[6], d[7])));
                    f[2] = __builtin_bit_cast(half8_t, make_uint4(codes_pair<2>(d[0], d[1]), codes_pair<2>(d[2], d[3]), codes_pair<2>(d[4], d[5]), codes_pair<2>(d[6], d[7])));
                    f[3] = __builtin_bit_cast(half8_t, make_uint4(codes_pair<3>(d[0], d[1]), codes_pair<3>(d[2], d[3]), codes_pair<3>(d[4], d[5]), codes_pair<3>(d[6], d[7])));
#pragma unroll
                    for (int k = 0; k < 4; k++)
#pragma unroll
                        for (int nb = 0; nb < NB; nb++)
#pragma unroll
                            for (int pt = 0; pt < kParts; pt++)
                                o[nb][4 * i + k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f[k], pf[nb][x][pt], o[nb][4 * i + k], 0, 0, 0);
                }
            }
            if (more) {
                load_v(tile + step);
                if (tile + 2 * step < stop) find_pages(tile + 2 * step);
            }
        }

        // join the waves: the column's sum first (a lane has summed its own positions)
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
            L[nb] += __shfl_xor(L[nb], 16);
            L[nb] += __shfl_xor(L[nb], 32);
            if (g == 0) {
                s_m[wave][16 * nb + n] = m[nb];
                s_e[wave][16 * nb + n] = E[nb];
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
        // four values of row r, from value d on, to o
        auto finish = [&](int r, int d, const float v[4], float E, float L) {
            const float inv = L > 0.0f ? 1.0f / L : 0.0f;
            float y[4];
#pragma unroll
            for (int i = 0; i < 4; i++) y[i] = ldexpf(v[i] * inv, (int)E + kCodeExp - kProbExp);
            int token, head;
            row_at(r, token, head);
            const int64_t off = ((q.first + token) * a.hq + head) * D + d;
            if constexpr (BF16) {
                uint2 u;
                u.x = pack_bf16(y[0], y[1]);
                u.y = pack_bf16(y[2], y[3]);
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.o) + off) = u;
            } else {
                *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + off) = make_float4(y[0], y[1], y[2], y[3]);
            }
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
                    const int i = 64 * y + lane, ir = i / (D / 4), id = 4 * (i % (D / 4)), r = x * kSumRows + ir;
                    const float4 f = *reinterpret_cast<const float4 *>(s_o + (wave * kSumRows + ir) * Lay::kRow + id);
                    const float v[4] = {f.x, f.y, f.z, f.w};
                    if (r < nrows) finish(r, id, v, s_e[wave][r], s_l[wave][r]);
                }
                sync();
            }
            at = unit1;
            continue;
        }
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
            const int r = 16 * nb + n;
            float mm = s_m[0][r], ee = kLow;
            for (int x = 1; x < kWaves; x++) mm = fmaxf(mm, s_m[x][r]);
            for (int x = 0; x < kWaves; x++) ee = fmaxf(ee, s_e[x][r] + (s_m[x][r] - mm));
            if (wave == nb && g == 0) {
                float l = 0.0f;
                for (int x = 0; x < kWaves; x++) l += s_l[x][r] * pow2_down(s_m[x][r] - mm);
                s_all[r] = make_float4(mm, ee, l, 0.0f);
            }
            const float q = pow2_down((m[nb] - mm) + (E[nb] - ee));
#pragma unroll
            for (int i = 0; i < kT; i++) o[nb][i] *= q;
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
                const float4 f = s_all[q0 + ir];
                st[x] = State{f.x, f.y, f.z};
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
                if (r < nrows) finish(r, id, v[x], st[x].E, st[x].L);
            }
        }
        at = unit1;
    }
}

template <int D, int NB>
int wgs_of(int num_cu) { return kPerCu<NB> * num_cu; }

template <int D, int NB>
hipError_t launch_nb(const AttnArgs &a, int bf16, int num_cu, hipStream_t stream) {
    const int wgs = wgs_of<D, NB>(num_cu);
    // at head_dim 256 the registers do not hold what both ways need (512 x 500 tokens of 24 / 4 heads 156 us, 128 without)
    if constexpr (NB == 1 && D < 256) {
        if (a.s.B * a.c.kv_heads >= (int64_t)wgs * kWaves) {
            if (bf16) k_attn_split<D, NB, true, true><<<wgs, kThreads, 0, stream>>>(a, wgs);
            else k_attn_split<D, NB, false, true><<<wgs, kThreads, 0, stream>>>(a, wgs);
            return hipGetLastError();
        }
    }
    if (bf16) k_attn_split<D, NB, true, false><<<wgs, kThreads, 0, stream>>>(a, wgs);
    else k_attn_split<D, NB, false, false><<<wgs, kThreads, 0, stream>>>(a, wgs);
    return hipGetLastError();
}

template <int D>
int64_t bytes_d(int num_cu) {
    const int64_t one = 2 * (int64_t)wgs_of<D, 1>(num_cu) * Layout<D, 1>::kRecord;
    const int64_t two = 2 * (int64_t)wgs_of<D, 2>(num_cu) * Layout<D, 2>::kRecord;
    return 4 * (one > two ? one : two);
}

}  // namespace

int64_t attn_split_bytes(int head_dim, int num_cu) {
    return head_dim == 64 ? bytes_d<64>(num_cu) : head_dim == 128 ? bytes_d<128>(num_cu) : bytes_d<256>(num_cu);
}

hipError_t launch_attn_split(const AttnArgs &a, int bf16, int blocks, int num_cu, hipStream_t stream) {
    switch (a.c.head_dim) {
        case 64: return blocks == 1 ? launch_nb<64, 1>(a, bf16, num_cu, stream) : launch_nb<64, 2>(a, bf16, num_cu, stream);
        case 128: return blocks == 1 ? launch_nb<128, 1>(a, bf16, num_cu, stream) : launch_nb<128, 2>(a, bf16, num_cu, stream);
        default: return blocks == 1 ? launch_nb<256, 1>(a, bf16, num_cu, stream) : launch_nb<256, 2>(a, bf16, num_cu, stream);
    }
}

}  // namespace w4a8
