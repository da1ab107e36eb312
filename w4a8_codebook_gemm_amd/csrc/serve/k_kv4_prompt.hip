// Attention over the paged cache in 4 bits for many query rows a sequence (prompts, their chunks).
//
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp2(s_t - m),  s_t = scale log2(e) q . k_t
//
// Matrix-core bound: 4 D flops for each row and position.  Units, waves and products are the int8
// cache's (k_attn_prompt.hip): blocks of 32 kWaves rows, 32 of them a wave's as the columns of
// v_mfma_f32_32x32x16_f16, queries and O^T in registers,
//   S^T [32 positions x 32 rows] = K Q^T,   O^T [D x 32] += V^T P^T,
// and a tile of 8192 / D positions becomes fp16 once for all waves, in LDS, two tiles deep, exactly
// (kv4_tiles.h).  V lies transposed as rows of values, its positions in the order in which a lane of
// S^T holds them, 4 (lane / 32) + 8 b + c, so probabilities never leave their lane.
//
// Scales are in the fragments and a head's unit is a factor of its scores and of its output, so a
// score is one multiply-add and one exponential, and the only statistic is the running maximum m, a
// whole number: rescaling is exact.
//
// Split: as in the other kernels, the tiles of all units form one line that is cut evenly over the
// workgroups; a cut unit's pieces are joined two and two in a tree.
//
// Measured (TFLOP/s of the positions that are seen; the library's product of 8192^3 reaches 1036 in fp16 here; the int8 kernel
// in brackets): 2 x 2048 tokens on 14000, 24 / 4 heads of 256, 1.40 to 1.44 ms, 1070 to 1100 (1.51); 8192 causal tokens, 32 / 8
// of 128, 577 to 590 us, 930 to 950 (609), 16 / 16 of 64 200, 685 (224); 5 ragged prompts of 128 160, 715 (163); fp32, which
// has twice the products, 2 x 2048 on 6000 of 128 770, 610 (822), 2 x 1024 on 2000 of 256 322 to 330, 380 (371).  The matrix
// cores are busy 43% of the cycles at head_dim 256, the vector units 49%: a SIMD's two waves take turns.  At
// head_dim 64 the softmax has four times the share.  At head_dim 256 bf16 spills 42 registers, outside
// the loop over tiles.
#include "kv4_tiles.h"

namespace w4a8 {
namespace {

typedef float floatx16 __attribute__((ext_vector_type(16)));

// What may move over the steps of the second product: vector and scalar arithmetic.  That and nothing: 8192 of 128 577 and 581
// us, 5 ragged ones 158 and 160, fp32 4096 of 64 91.2 and 94.2, bf16 8192 of 64 199.6 and 196.5.
constexpr int kSchedPV = 0x406;
// Tiles a workgroup is worth cutting for.  1, 4 and 8: 8 x 300 fresh tokens of 64 (32 / 8) 27.1, 26.9 and 30.6 us, of 128 36.6, 36.3 and
// 39.1, others alike.
constexpr int kMinTiles = 4;

template <int D, bool BF16>
struct Shape {
    // fp32 rows of 256 need the registers of two waves for their queries.  Two workgroups of 4 waves in place of one of 8 at
    // head_dim 64 and 128 pay where blocks of 128 rows are fuller: 20 x 100 with a window 35.2 and 30.0 us, 5 x 600 fp32 of 128
    // 69 and 64, 8192 of 64 200 and 224, of 128 594 and 676, 5 ragged ones 160 and 180.
    static constexpr int kWaves = BF16 || D <= 128 ? 8 : 4;
    static constexpr int kThreads = 64 * kWaves;
    static constexpr int RB = 32 * kWaves;
    static constexpr int T = 8192 / D;       // positions of a tile
    static constexpr int kGroups = T / 16;
    // see Line.  kOver 1, as it is, and 10 (kTail 1, as it is, 6): 8192 of 128 645, 577 and 574 us, 5 ragged ones 186, 158 and
    // 171, 8192 of 64 203, 200 and 216, fp32 4096 of 64 87.9, 91.2 and 110.7.
    static constexpr int kOver = D == 256 ? 5 : 3, kTail = D == 256 ? 3 : 2;
    static constexpr int kRegs = D / 2;      // floats of O^T in a lane
    static constexpr int kWaveRecord = 64 * (kRegs + 4);    // a wave's piece: O^T, then m, L
    static constexpr int kRecord = kWaves * kWaveRecord;
};

// The tiles in LDS.  Rows are 16 bytes longer than their values, so that the same 16-byte place of
// eight consecutive rows touches all banks, and every fragment is one address plus a constant.
//   K: a row for each position; its slot of 8 values x is at place x / 4 + (x % 4) (D / 32): a staging
//      thread writes four slots that follow each other, its neighbour the next four.
//   V: row d / 8 + (d % 8) (D / 8) for value d (a staging thread writes eight values, its neighbour the
//      next eight); place g has the positions 16 (g / 2) + 4 (g % 2) + {0..3, 8..11}, four a staging thread's.
template <int D>
struct Tile {
    static constexpr int kRow = 2 * D + 16, kBytes = 8192 / D * kRow;
    static constexpr int vRow = 16384 / D + 16, vBytes = D * vRow;
    static __device__ __forceinline__ int k_at(int t, int place) { return t * kRow + place * 16; }
    static __device__ __forceinline__ int v_at(int row, int place) { return row * vRow + place * 16; }
    // the first value that step s of the first product takes in half hh of the wave: place s + hh (D / 16)
    static __device__ __forceinline__ int q_at(int s, int hh) { return 32 * (s % (D / 32)) + 8 * (s / (D / 32)) + 16 * hh; }
};

// What sequence b0 + lane has: units, their tiles, the longest one's.  Called by whole waves: sequences of many blocks
// are summed by all lanes together.
struct Units {
    int64_t tiles;
    int units, longest;
};
template <class S>
__device__ __forceinline__ Units seq_units(const Attn4Args &a, int64_t b0, int lane) {
    Seq q{0, 0, 0, 0};
    if (b0 + lane < a.s.B) q = load_seq(a.s, a.M, a.page_shift, b0 + lane);
    const int64_t blocks = blocks_of<S>(a, q);
    int64_t tiles = 0;
    int longest = 0, x;
    auto add = [&](const Seq &r, int64_t i, int64_t &sum, int &most) {
        const int c = block_tiles<S>(a, r, i, x);
        sum += c;
        most = most > c ? most : c;
    };
    for (int64_t i = 0; i < (blocks <= 4 ? blocks : 0); i++) add(q, i, tiles, longest);
    for (uint64_t many = __ballot(blocks > 4); many; many &= many - 1) {
        const int src = __ffsll((unsigned long long)many) - 1;
        const Seq r = {0, lane_value(q.n, src), lane_value(q.len, src), lane_value(q.pos0, src)};
        const int64_t rb = blocks_of<S>(a, r);
        int64_t sum = 0;
        int most = 0;
        for (int64_t i = lane; i < rb; i += 64) add(r, i, sum, most);
        sum = lane_value(scan64(sum), 63);
        if (lane == src) tiles = sum;
        longest = longest > most ? longest : most;  // (whichever lane has it)
    }
    return Units{tiles * a.c.kv_heads, (int)blocks * a.c.kv_heads, longest};
}

template <int D, bool BF16>
__global__ __launch_bounds__((Shape<D, BF16>::kThreads), (Shape<D, BF16>::kWaves / 4)) void k_kv4_prompt(Attn4Args a, int wgs) {
    using S = Shape<D, BF16>;
    constexpr int kFrags = 2;  // K and V fragments in flight (2 and 4: alike)
    constexpr int T = S::T, kParts = BF16 ? 1 : 2, kSteps = D / 16, kTiles = D / 32;
    constexpr int kSubs = D == 256 ? 1 : 2, kWide = 32 * kSubs;   // positions of a softmax step: registers
    constexpr int kItems = 512 / S::kThreads;  // staging items of a thread: 256 of keys, 256 of values
    using L4 = Tile<D>;
    __shared__ __attribute__((aligned(16))) char s_k[2][L4::kBytes], s_v[2][L4::vBytes];
    __shared__ int s_there[2][S::kGroups];  // of each group of 16 positions: whether its page is there
    __shared__ int64_t s_mine[64], s_incl[64];  // tiles of the only 64 sequences, and up to each
    __shared__ int s_flag;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), n = lane & 31, hh = lane >> 5;
    uint32_t *counters = static_cast<uint32_t *>(a.ws);
    float *pieces = reinterpret_cast<float *>(static_cast<char *>(a.ws) + kAttnCounterBytes);

    int64_t line = 0, incl_line = 0, units = 0;
    int incl_units = 0, longest = 0;  // (64 sequences have fewer than 2^30 units)
    Units u{0, 0, 0};
    for (int64_t b0 = 0; b0 < a.s.B; b0 += 64) {
        u = seq_units<S>(a, b0, lane);
        incl_units = scan32(u.units);
        incl_line = scan64(u.tiles + (int64_t)S::kOver * u.units);
        units += lane_value(incl_units, 63);
        line += lane_value(incl_line, 63);
        longest = longest > u.longest ? longest : u.longest;
    }
    if (line == 0) return;
    int64_t used = (line + kMinTiles - 1) / kMinTiles;
    if (used > wgs) used = wgs;
    // Whole units, one a workgroup and a place on the line each, where workgroups are enough and the longest is no more than a cut's
    // part: it joins nothing.  Cut and whole (us): 5 x 600 fresh tokens (16 / 16 heads of 64) 27.3 and 20.8, 30 x 20 on 500 (32 / 8 of
    // 128) 29.2 and 21.5, fp32 36.6 and 28.7.  Finding out costs the others 0.3 us.
    const bool whole = units <= wgs && max_lanes(longest) <= div64(line, used);
    if (whole) line = used = units;
    auto places = [&](const Units &x) { return whole ? x.units : x.tiles + (int64_t)S::kOver * x.units; };
    if (a.s.B <= 64) {  // every wave writes the same and reads its own
        s_mine[lane] = places(u);
        s_incl[lane] = whole ? incl_units : incl_line;
    }
    // workgroups go to the XCDs in turn: neighbours on the line, which read the same pages, share one's L2
    int64_t w = blockIdx.x;
    if (used == wgs && wgs % 8 == 0) w = w % 8 * (wgs / 8) + w / 8;
    if (w >= used) return;
    const Line cut{line, used, S::kOver, S::kTail};
    const int64_t t1 = cut.begin(w + 1);

    int64_t from = 0, from_base = 0;  // the 64 sequences that the last unit was in, and their place
    for (int64_t at = cut.begin(w); at < t1;) {
        // the sequence, cache head and row block that tile `at` is in
        int64_t base = from_base, b = 0, per_head = 0;
        for (int64_t b0 = from; b0 < a.s.B; b0 += 64) {
            const int64_t mine = a.s.B <= 64 ? s_mine[lane] : places(seq_units<S>(a, b0, lane));
            const int64_t incl = a.s.B <= 64 ? s_incl[lane] : scan64(mine);
            const int64_t sum = lane_value(incl, 63);
            if (at < base + sum) {
                const int src = __ffsll((unsigned long long)__ballot(at - base < incl)) - 1;
                from = b0;
                from_base = base;
                b = b0 + src;
                base += lane_value(incl - mine, src);
                per_head = div64(lane_value(mine, src), a.c.kv_heads);
                break;
            }
            base += sum;
        }
        const Seq q = load_seq(a.s, a.M, a.page_shift, b);
        const int64_t blocks = blocks_of<S>(a, q);
        const int h = (int)div64(at - base, per_head);
        int64_t unit0 = base + h * per_head, rb = 0;  // the unit's first tile on the line
        int first_tile = 0, tiles = 1;
        for (int64_t r = 0; r < blocks; r += 64) {
            int f = 0, c = 0;
            if (r + lane < blocks) c = block_tiles<S>(a, q, r + lane, f);
            const int64_t place = r + lane < blocks ? (whole ? 1 : c + S::kOver) : 0;
            const int64_t incl = scan64(place), sum = lane_value(incl, 63);
            if (at < unit0 + sum) {
                const int src = __ffsll((unsigned long long)__ballot(at - unit0 < incl)) - 1;
                unit0 += lane_value(incl - place, src);
                rb = r + src;
                first_tile = lane_value(f, src);
                tiles = lane_value(c, src);
                break;
            }
            unit0 += sum;
        }
        const int64_t unit1 = unit0 + (whole ? 1 : S::kOver + tiles);
        int tile0 = 0, tile1 = tiles;
        if (!whole && !cut.part(at, t1, unit0, unit1, tiles, tile0, tile1)) {
            at = unit1;
            continue;
        }

        // this wave's rows
        const int64_t rows = (int64_t)q.n * a.group, r0 = rb * S::RB + 32 * wave;
        const int nrows = rows - r0 < 0 ? 0 : rows - r0 < 32 ? (int)(rows - r0) : 32;
        // the row's token and head, found again where they are wanted: registers are what the loop lacks
        auto row_of = [&](int64_t &token, int &head) {
            const int l = fresh(lane) & 31;
            const int64_t my = r0 + (l < nrows ? l : 0);
            token = div64(my, a.group);
            head = h * a.group + (int)(my - token * a.group);
        };
        int hi = 0, all_lo = 0, all_hi = 0, any_lo = 0, any_hi = 0;
        if (nrows) {
            int64_t token;
            int x;
            row_of(token, x);
            if (n < nrows) sees(a, q, token, x, hi);
            sees(a, q, div64(r0, a.group), any_lo, all_hi);
            sees(a, q, div64(r0 + nrows - 1, a.group), all_lo, any_hi);
        }
        half8_t qf[kParts][kSteps];
        float fac;
        {
            float top = 0.0f;
            int64_t token = 0;
            int head = 0;
            if (nrows) row_of(token, head);
            // (a wave without rows reads the first row of its sequence, for nothing)
            const int64_t off = (q.first + token) * a.q_stride + (int64_t)head * D;
            int k_exp;
            const float k_part = frexpf(a.c.k_unit[h], &k_exp);
            // all of the row's values at once, as they lie
            RawQ<BF16> raw[kSteps];
#pragma unroll
            for (int s = 0; s < kSteps; s++) raw[s].load(a.q, off + L4::q_at(s, hh));
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int s = 0; s < kSteps; s++) {
                float v[8];
                raw[s].values(v);
#pragma unroll
                for (int i = 0; i < 8; i++) top = fmaxf(top, fabsf(v[i]));
            }
            if (n >= nrows) top = 0.0f;
            top = max_xor32(top);
            // the row's largest value at 2^13 .. 2^14, as in the split kernel
            int ex = 0;
            if (top > 0.0f) frexpf(top, &ex);
            fac = fmaxf(ldexpf(fabsf(a.scale) * kLog2e * k_part, ex + k_exp - 14 + kValueExp), 0x1p-126f);
#pragma unroll
            for (int s = 0; s < kSteps; s++) {
                float v[8];
                raw[s].values(v);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    v[i] = n < nrows ? ldexpf(a.scale < 0.0f ? -v[i] : v[i], 14 - ex) : 0.0f;
                    qf[0][s][i] = (_Float16)v[i];
                    if constexpr (kParts == 2) qf[1][s][i] = (_Float16)(v[i] - (float)(_Float16)v[i]);
                }
            }
        }
        floatx16 o[kTiles];
#pragma unroll
        for (int i = 0; i < kTiles; i++) o[i] = floatx16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
        float m = kLow, L = 0.0f;

        // staging: item i < 256 holds 8 values of 4 positions of V, the others 32 values of a position of K
        const int P = a.c.page_size, pm = P - 1;
        const int32_t *table = a.s.page_table + b * a.s.table_width;
        uint32_t st[kItems][4], sc[kItems];  // codes, scale bytes
        int st_there = 0;
        int page[kItems];
        auto item_v = [&](int i) { return S::kWaves == 8 ? wave < 4 : i == 0; };
        // V: group of four positions, eight values; K: position, chunk
        auto place_v = [&](int &vg, int &vd) {
            const int it = fresh(tid) & 255;
            vg = it / (D / 8);
            vd = it % (D / 8);
        };
        auto place_k = [&](int &kt, int &kc) {
            const int it = fresh(tid) & 255;
            kt = it / (D / 32);
            kc = it % (D / 32);
        };
        auto teller = [&]() { return (fresh(tid) & 255) % (D / 2) == 0; };  // says whether 16 positions' page is there
        auto find_page = [&](int tile, int i) {
            int x, y;
            if (item_v(i)) {
                place_v(x, y);
                x = 4 * x;
            } else {
                place_k(x, y);
            }
            const int t = tile * T + x;
            return t < q.len ? table[t >> a.page_shift] : -1;
        };
        auto load = [&](int tile) {
#pragma unroll
            for (int i = 0; i < kItems; i++) {
                const bool ok = (uint32_t)page[i] < (uint32_t)a.c.num_pages;
                const int64_t blk = (int64_t)(ok ? page[i] : 0) * a.c.kv_heads + h;
                if (item_v(i)) {
                    int vg, vd;
                    place_v(vg, vd);
                    const int slot = (tile * T + 4 * vg) & pm;
                    const uint8_t *p = a.c.v + (blk * P + slot) * (D / 2) + 4 * vd;
#pragma unroll
                    for (int j = 0; j < 4; j++) st[i][j] = *reinterpret_cast<const uint32_t *>(p + j * (D / 2));
                    sc[i] = *reinterpret_cast<const uint32_t *>(a.c.v_scale + (blk * (D / 16) + (vd >> 1)) * P + slot);
                    st_there = ok;
                } else {
                    int kt, kc;
                    place_k(kt, kc);
                    const int64_t row = blk * P + ((tile * T + kt) & pm);
                    const uint4 x = *reinterpret_cast<const uint4 *>(a.c.k + row * (D / 2) + 16 * kc);
                    st[i][0] = x.x; st[i][1] = x.y; st[i][2] = x.z; st[i][3] = x.w;
                    sc[i] = *reinterpret_cast<const uint16_t *>(a.c.k_scale + row * (D / 16) + 2 * kc);
                }
            }
        };
        auto store = [&](int buf) {
#pragma unroll
            for (int i = 0; i < kItems; i++) {
                if (item_v(i)) {
                    int vg, vd;
                    place_v(vg, vd);
                    // four positions are half a place
                    char *p = s_v[buf] + L4::v_at(vd, 2 * (vg >> 2) + (vg & 1)) + (vg & 2) * 4;
                    const half2_t s0 = scale_pair<0>(sc[i]), s1 = scale_pair<2>(sc[i]);
                    const uint32_t e0 = even_codes(st[i][0], st[i][1]), e1 = even_codes(st[i][2], st[i][3]);
                    const uint32_t d0 = odd_codes(st[i][0], st[i][1]), d1 = odd_codes(st[i][2], st[i][3]);
                    auto row = [&](int y, uint32_t first, uint32_t second) {  // value 8 vd + y
                        *reinterpret_cast<uint2 *>(p + L4::v_at(y * (D / 8), 0)) = make_uint2(first, second);
                    };
                    row(0, codes_times<0>(e0, s0), codes_times<0>(e1, s1));
                    row(1, codes_times<0>(d0, s0), codes_times<0>(d1, s1));
                    row(2, codes_times<1>(e0, s0), codes_times<1>(e1, s1));
                    row(3, codes_times<1>(d0, s0), codes_times<1>(d1, s1));
                    row(4, codes_times<2>(e0, s0), codes_times<2>(e1, s1));
                    row(5, codes_times<2>(d0, s0), codes_times<2>(d1, s1));
                    row(6, codes_times<3>(e0, s0), codes_times<3>(e1, s1));
                    row(7, codes_times<3>(d0, s0), codes_times<3>(d1, s1));
                    if (teller()) s_there[buf][vg >> 2] = st_there;
                } else {
                    int kt, kc;
                    place_k(kt, kc);
                    char *p = s_k[buf] + L4::k_at(kt, kc);
                    const half2_t s0 = scale_both<0>(sc[i]), s1 = scale_both<1>(sc[i]);
#pragma unroll
                    for (int x = 0; x < 4; x++)
                        *reinterpret_cast<half8_t *>(p + L4::k_at(0, x * (D / 32))) = values_natural(st[i][x], x < 2 ? s0 : s1);
                }
            }
        };

        const int begin = first_tile + tile0, end = first_tile + tile1;
#pragma unroll
        for (int i = 0; i < kItems; i++) page[i] = find_page(begin, i);
        load(begin);
#pragma unroll
        for (int i = 0; i < kItems; i++) page[i] = begin + 1 < end ? find_page(begin + 1, i) : -1;
        store(0);
        __syncthreads();
        for (int tile = begin; tile < end; tile++) {
            const int buf = (tile - begin) & 1;
            if (tile + 1 < end) {
                load(tile + 1);
#pragma unroll
                for (int i = 0; i < kItems; i++) page[i] = tile + 2 < end ? find_page(tile + 2, i) : -1;
            }
#pragma unroll 1
            for (int step = 0; step < T / kWide; step++) {
                const int p0 = tile * T + kWide * step;
                if (p0 >= any_hi || any_lo - p0 >= kWide) continue;  // uniform over the wave
                int there[kWide / 16];
#pragma unroll
                for (int u = 0; u < kWide / 16; u++) there[u] = s_there[buf][step * (kWide / 16) + u];
                const int ln = fresh(lane);
                const char *kp = s_k[buf] + L4::k_at(kWide * step + (ln & 31), (ln >> 5) * (D / 16));
                const char *vp = s_v[buf] + L4::v_at(ln & 31, 2 * (kWide / 16) * step + (ln >> 5));
                auto k_frag = [&](int x) {  // step x % kSteps of positions 32 (x / kSteps) ..
                    return *reinterpret_cast<const half8_t *>(kp + L4::k_at(32 * (x / kSteps), x % kSteps));
                };
                auto v_frag = [&](int x) {  // values 32 (x % kTiles) .., positions 16 (x / kTiles) ..
                    return *reinterpret_cast<const half8_t *>(vp + L4::v_at(32 * (x % kTiles), 2 * (x / kTiles)));
                };
                floatx16 s[kSubs];
#pragma unroll
                for (int y = 0; y < kSubs; y++) s[y] = floatx16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
                half8_t kf[kFrags];
#pragma unroll
                for (int x = 0; x < kFrags; x++) kf[x] = k_frag(x);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int x = 0; x < kSubs * kSteps; x++) {
                    const half8_t k = kf[x % kFrags];
                    if (x + kFrags < kSubs * kSteps) kf[x % kFrags] = k_frag(x + kFrags);
                    const int i = x % kSteps, y = x / kSteps;
#pragma unroll
                    for (int pt = 0; pt < kParts; pt++) s[y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, qf[pt][i], s[y], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                }
                half8_t vf[kFrags];
#pragma unroll
                for (int x = 0; x < kFrags; x++) vf[x] = v_frag(x);
                __builtin_amdgcn_sched_barrier(0);
                int every = there[0];
#pragma unroll
                for (int u = 1; u < kWide / 16; u++) every &= there[u];
                if (!(p0 >= all_lo && all_hi - p0 >= kWide && every)) {
                    const int to = hi - p0 - 4 * (ln >> 5), from = a.window ? __builtin_elementwise_sub_sat(to, (int)a.window) : -p0 - kWide;
#pragma unroll
                    for (int j = 0; j < 16 * kSubs; j++) {
                        const int t = 8 * (j >> 2) + (j & 3);
                        const bool see = (t >= from) & (t < to) & (there[j >> 3] != 0);
                        s[j >> 4][j & 15] = see ? s[j >> 4][j & 15] : -INFINITY;
                    }
                }
                float top = s[0][0];
#pragma unroll
                for (int j = 1; j < 16 * kSubs; j++) top = fmaxf(top, s[j >> 4][j & 15]);
                top = max_xor32(top);
                const float mn = running_maximum(m, top * fac);
                const float down = m - mn;
                if (__any(down < 0.0f)) {
                    const float x = pow2_down(down);
                    L *= x;
#pragma unroll
                    for (int i = 0; i < kTiles; i++) o[i] *= x;
                }
                m = mn;
                const float c = (float)kProbExp - mn;
                half8_t pf[2 * kSubs][kParts];  // positions 16 x .. of the step
                auto weights = [&](int y) {     // of its 32 positions 32 y ..
                    float sum = 0.0f;
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float p0x = __builtin_amdgcn_exp2f(fmaf(s[y][j], fac, c));   // 2^14 at most
                        const float p1x = __builtin_amdgcn_exp2f(fmaf(s[y][j + 1], fac, c));
                        sum += p0x + p1x;
                        const int z = 2 * y + (j >> 3);
                        if constexpr (BF16) {
                            pf[z][0][j & 7] = (_Float16)p0x;
                            pf[z][0][(j & 7) + 1] = (_Float16)p1x;
                        } else {
                            float minus = -1.0f;
                            asm("" : "+v"(minus));   // fma takes an fp16 number as it is, a subtraction would widen it first
                            uint32_t hw = pack_half(p0x, p1x);
                            asm("" : "+v"(hw));      // once: what is taken off is what was kept
                            const half2_t hp = __builtin_bit_cast(half2_t, hw);
                            pf[z][0][j & 7] = hp[0];
                            pf[z][0][(j & 7) + 1] = hp[1];
                            pf[z][kParts - 1][j & 7] = (_Float16)fmaf((float)hp[0], minus, p0x);
                            pf[z][kParts - 1][(j & 7) + 1] = (_Float16)fmaf((float)hp[1], minus, p1x);
                        }
                    }
                    L += sum;
                };
                weights(0);
                __builtin_amdgcn_sched_barrier(kSchedPV);
#pragma unroll
                for (int x = 0; x < 2 * kSubs * kTiles; x++) {
                    if (kSubs == 2 && x == 2 * kTiles) weights(kSubs - 1);
                    const half8_t v = vf[x % kFrags];
                    if (x + kFrags < 2 * kSubs * kTiles) vf[x % kFrags] = v_frag(x + kFrags);
#pragma unroll
                    for (int pt = 0; pt < kParts; pt++)
                        o[x % kTiles] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, pf[x / kTiles][pt], o[x % kTiles], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(kSchedPV);
                }
            }
            if (tile + 1 < end) store(buf ^ 1);
            __syncthreads();
        }
        L += __shfl_xor(L, 32);

        bool write = true;
        if (tile1 - tile0 < tiles) {
            const int64_t w_first = cut.first(unit0), w_end = cut.last(unit1);
            auto slot = [&](unsigned x) {
                return shared_piece(pieces + (2 * (w_first + x) + (x == 0 ? 1 : 0)) * S::kRecord + wave * S::kWaveRecord, 4 * S::kWaveRecord);
            };
            unsigned held = (unsigned)(w - w_first);
            write = join_pieces<2>(counters, w_first, w, w_end, &s_flag, [&](unsigned x) {
                if (nrows == 0) return;
                const __amdgpu_buffer_rsrc_t p = slot(x);
#pragma unroll
                for (int i = 0; i < S::kRegs / 4; i++)
                    put_shared4(p, i * 1024 + lane * 16, o[i >> 2][4 * (i & 3)], o[i >> 2][4 * (i & 3) + 1], o[i >> 2][4 * (i & 3) + 2], o[i >> 2][4 * (i & 3) + 3]);
                put_shared4(p, S::kRegs * 256 + lane * 16, m, L, 0.0f, 0.0f);
            }, [&](unsigned x, unsigned step, unsigned) {
                // of the node's two slots this workgroup holds one; a sum of two does not ask for their order
                if (nrows == 0) return;
                const __amdgpu_buffer_rsrc_t p = slot(held == x ? x + step : x);
                held = x;
                const floatx4 other = get_shared4(p, S::kRegs * 256 + lane * 16);
                constexpr int kAtOnce = S::kRegs / 4 < 16 ? S::kRegs / 4 : 16;  // 16-byte loads in flight
                float qa = 0.0f, qb = 0.0f;
#pragma unroll
                for (int i0 = 0; i0 < S::kRegs / 4; i0 += kAtOnce) {
                    floatx4 v[kAtOnce];
#pragma unroll
                    for (int i = 0; i < kAtOnce; i++) v[i] = get_shared4(p, (i0 + i) * 1024 + lane * 16);
                    __builtin_amdgcn_sched_barrier(0);
                    if (i0 == 0) {
                        const State t = join(State{m, 0.0f, L}, State{other[0], 0.0f, other[1]}, qa, qb);
                        m = t.m;
                        L = t.L;
                    }
#pragma unroll
                    for (int i = 0; i < 4 * kAtOnce; i++) {
                        const int r = 4 * i0 + i;
                        o[r >> 4][r & 15] = o[r >> 4][r & 15] * qa + v[i >> 2][i & 3] * qb;
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            });
        }
        if (write && n < nrows) {
            // the sum of the probabilities carries the same 2^14 as the products
            int v_exp;
            const float v_part = frexpf(a.c.v_unit[h], &v_exp), inv = L > 0.0f ? v_part / L : 0.0f;
            int64_t token;
            int head;
            row_of(token, head);
            const int64_t off = ((q.first + token) * a.hq + head) * D;
            // value 8 x + y is in row x + y (D / 8) of O^T; this lane has the rows 32 i + 8 j + 4 hh + c
#pragma unroll
            for (int z = 0; z < D / 16; z++) {
                const int x = (z >> 2) * 8 + (z & 3);   // and + 4 hh
                float v[8];
#pragma unroll
                for (int y = 0; y < 8; y++) {
                    const int row = x + y * (D / 8);
                    v[y] = ldexpf(o[row >> 5][((row & 31) >> 3) * 4 + (row & 3)] * inv, v_exp + kValueExp);
                }
                const int64_t d = off + 8 * (x + 4 * hh);
                if constexpr (BF16) {
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.o) + d) =
                        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
                } else {
                    float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(a.o) + d);
                    p[0] = make_float4(v[0], v[1], v[2], v[3]);
                    p[1] = make_float4(v[4], v[5], v[6], v[7]);
                }
            }
        }
        at = unit1;
    }
}

template <int D>
hipError_t launch_d(const Attn4Args &a, int bf16, int num_cu, hipStream_t stream) {
    if (bf16) k_kv4_prompt<D, true><<<num_cu, Shape<D, true>::kThreads, 0, stream>>>(a, num_cu);
    else k_kv4_prompt<D, false><<<num_cu, Shape<D, false>::kThreads, 0, stream>>>(a, num_cu);
    return hipGetLastError();
}

}  // namespace

int64_t kv4_prompt_bytes(int head_dim, int num_cu) {
    const int64_t regs = head_dim / 2;
    return 4 * 2 * (int64_t)num_cu * 8 * 64 * (regs + 4);
}

hipError_t launch_kv4_prompt(const Attn4Args &a, int bf16, int num_cu, hipStream_t stream) {
    switch (a.c.head_dim) {
        case 64: return launch_d<64>(a, bf16, num_cu, stream);
        case 128: return launch_d<128>(a, bf16, num_cu, stream);
        default: return launch_d<256>(a, bf16, num_cu, stream);
    }
}

}  // namespace w4a8
