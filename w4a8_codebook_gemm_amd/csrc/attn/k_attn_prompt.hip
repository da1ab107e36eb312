// Attention over the int8 paged cache for many query rows a sequence (prompts, their chunks).
//
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp2(s_t - m),  s_t = scale log2(e) q . k_t
//
// Matrix-core bound: 4 D flops for each row and position.  A unit is a block of 32 kWaves rows (the
// (token, query head) pairs of one sequence and cache head); each wave has 32 of them as the
// columns of v_mfma_f32_32x32x16_f16, queries and O^T in registers:
//   S^T [32 positions x 32 rows] = K Q^T,   O^T [D x 32] += V^T P^T.
// The codes of a tile of 8192 / D positions become fp16 once for all waves, in LDS, two tiles
// deep: loads of the next tile are in flight while this one is used.  K lies as rows of
// positions, V transposed as rows of values (a permute picks one value of two positions), both in
// 16-byte slots placed so that eight neighbouring lanes touch all banks in reading and in writing.
// V's positions are kept in the order in which a lane of S^T holds them, 4 (lane / 32) + 8 b + c,
// so probabilities never leave their lane.
//
// Pages hold at least 16 positions, so the scales are the same for the 16 positions of a group.
// The running maximum m and the exponent E are whole numbers as in the split kernel:
// a probability enters the second product as p w, w = sv 2^(14 - E), at most 2^14.  With bf16
// outputs the factor goes into the exponent, p w = exp2(s + (log2 w - m)): log2 w is good to 2^-18 for
// |log2 w| <= 60, and log2 w - m is rounded at m's size, half a step, which is 2^-24 |m| at most and
// what the score itself is off by.  (w as a factor of p, as the split kernel has it, is free of that and
// takes 1 to 6% longer: 8192 tokens, 32 / 8 heads of 128, 642 and 625 us, heads of 64 471 and 443.)  w is
// held at 2^-60 or more, where the products are below fp16's range and only the sum of p counts them.
//
// Split: as in the split kernel, the tiles of all units form one line that is cut evenly over the
// workgroups; a cut unit's pieces are joined two and two in a tree.
//
// Measured (TFLOP/s of the positions that are seen; the library's large fp16 product reaches 1125): 2 x 2048 tokens on
// 14000, 24 / 4 heads of 256, 1.46 to 1.55 ms, 940 to 1000; 8192 causal tokens, 32 / 8 of 128, 620 to 690 us, 800 to 890, of
// 256 (24 / 4) 910 to 940 us, 880 to 910, of 64 436 to 494 us, 560 to 630; 8192 of 128 without a mask 1150 to 1220 us, 900
// to 960.  fp32 has twice the products: 2 x 2048 on 6000, 32 / 8 of 128, 842 to 862 us, 550; 2 x 1024 on 2000, 24 / 4 of
// 256, 390 us, 320, with one wave a SIMD.  The matrix cores are busy 44% of the cycles at head_dim 256: both products and
// the softmax between them take turns on a SIMD's two waves, some 5 vector instructions a score.  At head_dim 64 a score
// has a quarter of the products: a step of 64 positions has some 185 vector instructions and 35 exponentials, 1300 cycles, to 512
// cycles of products, so 39% is the most that two waves in turn could keep busy.  It is 25%: the waves also wait.
// At head_dim 256 the bf16 kernels spill 44 to 46 registers (fp32 from 128 on 7 to 13): but for one, read in the loop over
// tiles, each unit pays once.
#include "attn_tiles.h"

namespace w4a8 {
namespace {

typedef float floatx16 __attribute__((ext_vector_type(16)));

// Query fragments of bf16 heads of 256 that stay in LDS.  None, 2 and 4: 2 x 2048 tokens on 14000 1547 to 1581, 1480
// to 1485 and 1508 to 1512 us.
constexpr int kQFar = 2;
// What the compiler may move over the steps of the second product: vector and scalar arithmetic, so that
// one half's weights fill the matrix core's time on the other's.
constexpr int kSchedPV = 0x406;
constexpr float kNoPage = 1e9f;
// Tiles a workgroup is worth cutting for.  1, 4 and 8: 100 tokens on 1000 (32 / 8 heads of 128) 31.9, 32.2 and 36.1 us, 8 x 100
// fresh ones 16.2, 17.5 and 26.2, longer calls alike.
constexpr int kMinTiles = 4;

template <int D, bool BF16>
struct Shape {
    // fp32 rows need twice the registers for their queries: at D 256 half the waves share a CU.  (D 128 with
    // 4 waves 1299 us for 2 x 2048 tokens on 6k, with two such workgroups 947, with 8 waves 862.)
    static constexpr int kWaves = BF16 || D <= 128 ? 8 : 4;
    static constexpr int kThreads = 64 * kWaves;
    static constexpr int RB = 32 * kWaves;
    static constexpr int T = 8192 / D;       // positions of a tile
    static constexpr int kGroups = T / 16;
    // see Line: a unit's start and end cost some 7 us, a tile 2 (D 256: 1.3).  kOver at 0, as it is, and at 10: 4096 tokens of
    // 24 / 4 heads of 256 384, 284 and 286 us, 8192 of 64 500, 436 and 477, 5 ragged prompts of 128 438, 402 and 415.  kTail at 1, as it is,
    // and at 6: 8192 of 64 445, 436 and 441, 100 on 1000 of 128 32.0, 32.2 and 36.0, 2 x 2048 on 14000 of 256 1502, 1482 and 1504.
    static constexpr int kOver = D == 256 ? 5 : 3, kTail = D == 256 ? 3 : 2;
    static constexpr int kRegs = D / 2;      // floats of O^T in a lane
    static constexpr int kWaveRecord = 64 * (kRegs + 4);    // a wave's piece: O^T, then m, E, L
    static constexpr int kRecord = kWaves * kWaveRecord;
};

// First tile and tiles of row block rb of a sequence.
template <int D, bool BF16>
__device__ __forceinline__ int block_tiles(const AttnArgs &a, const Seq &q, int64_t rb, int &first) {
    using S = Shape<D, BF16>;
    const int64_t rows = (int64_t)q.n * a.group, r0 = rb * S::RB;
    const int64_t last = (r0 + S::RB < rows ? r0 + S::RB : rows) - 1;
    int lo, hi, x;
    sees(a, q, div64(r0, a.group), lo, x);
    sees(a, q, div64(last, a.group), x, hi);
    first = lo / S::T;
    const int n = tiles_to<S::T>(hi) - first;
    return n < 1 ? 1 : n;  // rows that see nothing are still written
}

template <int D, bool BF16>
__device__ __forceinline__ int64_t blocks_of(const AttnArgs &a, const Seq &q) {
    return div64((int64_t)q.n * a.group + Shape<D, BF16>::RB - 1, Shape<D, BF16>::RB);
}

// Places of sequence b0 + lane on the line.  Called by whole waves: sequences of many blocks are
// summed by all lanes together.
template <int D, bool BF16>
__device__ __forceinline__ int64_t seq_tiles(const AttnArgs &a, int64_t b0, int lane) {
    Seq q{0, 0, 0, 0};
    if (b0 + lane < a.s.B) q = load_seq(a.s, a.M, a.page_shift, b0 + lane);
    const int64_t blocks = blocks_of<D, BF16>(a, q);
    int64_t tiles = 0;
    int x;
    for (int64_t i = 0; i < (blocks <= 4 ? blocks : 0); i++) tiles += block_tiles<D, BF16>(a, q, i, x) + Shape<D, BF16>::kOver;
    for (uint64_t many = __ballot(blocks > 4); many; many &= many - 1) {
        const int src = __ffsll((unsigned long long)many) - 1;
        const Seq r = {0, lane_value(q.n, src), lane_value(q.len, src), lane_value(q.pos0, src)};
        const int64_t rb = blocks_of<D, BF16>(a, r);
        int64_t sum = 0;
        for (int64_t i = lane; i < rb; i += 64) sum += block_tiles<D, BF16>(a, r, i, x) + Shape<D, BF16>::kOver;
        sum = lane_value(scan64(sum), 63);
        if (lane == src) tiles = sum;
    }
    return tiles * a.c.kv_heads;
}

// The tiles in LDS.  Rows are 16 bytes longer than their values, so that the same 16-byte slot of
// eight consecutive rows touches all banks, and every fragment is one address plus a constant.
//   K: a row for each position; its 8-value slots even ones first, then odd ones (a staging thread
//      writes a pair of them, its neighbour the next pair).
//   V: row d / 4 + (d % 4) (D / 4) for value d (a staging thread writes four values, its neighbour the
//      next four); slot g has the positions 16 (g / 2) + 4 (g % 2) + {0..3, 8..11}.  Row r of
//      O^T is then value v_value(r).
template <int D>
struct Tile {
    static constexpr int kRow = 2 * D + 16, kBytes = 8192 / D * kRow;
    static constexpr int vRow = 16384 / D + 16, vBytes = D * vRow;
    static __device__ __forceinline__ int k_at(int t, int slot) { return t * kRow + ((slot >> 1) + (slot & 1) * (D / 16)) * 16; }
    static __device__ __forceinline__ int v_row(int d) { return (d >> 2) + (d & 3) * (D / 4); }
    static __device__ __forceinline__ int v_at(int row, int slot) { return row * vRow + slot * 16; }
};

// kSmall: pages of 16 positions, else of 32 or more.
template <int D, bool BF16, bool kSmall>
__global__ __launch_bounds__((Shape<D, BF16>::kThreads), (Shape<D, BF16>::kWaves / 4)) void k_attn_prompt(AttnArgs a, int wgs) {
    using S = Shape<D, BF16>;
    // K and V fragments in flight.  2 and 4: at D 256 (2 x 2048 tokens on 14000) 1482 and 1660 us, at D 128 (8 x 64 on 2000)
    // 45.0 and 44.3, at D 64 436 and 436
    constexpr int kAhead = D == 128 ? 4 : 2;
    constexpr int T = S::T, kParts = BF16 ? 1 : 2, kSteps = D / 16, kTiles = D / 32;
    constexpr int kQLds = D == 256 && BF16 ? kQFar : 0;  // query fragments that stay in LDS
    constexpr int kSubs = D == 256 ? 1 : 2, kWide = 32 * kSubs;   // positions of a softmax step: registers
    constexpr int kSpan = kSmall ? 16 : 32;                       // positions that surely share a page
    constexpr int kScales = kWide / kSpan, kOf = kSpan / 2;       // pages of a step; a lane's scores of one
    constexpr int kItems = 512 / S::kThreads;  // staging items of a thread: 256 of keys, 256 of values
    using L8 = Tile<D>;
    __shared__ __attribute__((aligned(16))) char s_k[2][L8::kBytes], s_v[2][L8::vBytes];
    // of each group of 16 positions: key scale, value scale, its log2, its exponent (kNoPage: no such page)
    __shared__ float4 s_sc[2][S::kGroups];
    __shared__ __attribute__((aligned(16))) char s_q[kQLds ? kQLds * S::kThreads * 16 : 16];
    __shared__ int64_t s_mine[64], s_incl[64];  // tiles of the only 64 sequences, and up to each
    __shared__ int s_flag;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), n = lane & 31, hh = lane >> 5;
    uint32_t *counters = static_cast<uint32_t *>(a.ws);
    float *pieces = reinterpret_cast<float *>(static_cast<char *>(a.ws) + kAttnCounterBytes);

    int64_t line = 0;
    for (int64_t b0 = 0; b0 < a.s.B; b0 += 64) {
        const int64_t mine = seq_tiles<D, BF16>(a, b0, lane), incl = scan64(mine);
        line += lane_value(incl, 63);
        if (a.s.B <= 64) {  // every wave writes the same and reads its own
            s_mine[lane] = mine;
            s_incl[lane] = incl;
        }
    }
    if (line == 0) return;
    int64_t used = (line + kMinTiles - 1) / kMinTiles;
    if (used > wgs) used = wgs;
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
            const int64_t mine = a.s.B <= 64 ? s_mine[lane] : seq_tiles<D, BF16>(a, b0, lane);
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
        const int64_t blocks = blocks_of<D, BF16>(a, q);
        const int h = (int)div64(at - base, per_head);
        int64_t unit0 = base + h * per_head, rb = 0;  // the unit's first tile on the line
        int first_tile = 0, tiles = 1;
        for (int64_t r = 0; r < blocks; r += 64) {
            int f = 0, c = 0;
            if (r + lane < blocks) c = block_tiles<D, BF16>(a, q, r + lane, f);
            const int64_t place = r + lane < blocks ? c + S::kOver : 0;
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
        const int64_t unit1 = unit0 + S::kOver + tiles;
        int tile0, tile1;
        if (!cut.part(at, t1, unit0, unit1, tiles, tile0, tile1)) {
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
        half8_t qf[kParts][kSteps - kQLds];
        float fac;
        {
            float top = 0.0f;
            int64_t token = 0;
            int head = 0;
            if (nrows) row_of(token, head);
            // (a wave without rows reads the first row of its sequence, for nothing)
            const int64_t off = (q.first + token) * a.q_stride + (int64_t)head * D + 8 * hh;
            // all of the row's values at once, as they lie
            RawQ<BF16> raw[kSteps];
#pragma unroll
            for (int s = 0; s < kSteps; s++) raw[s].load(a.q, off + 16 * s);
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
            fac = ldexpf(fabsf(a.scale) * kLog2e, ex - 14);
#pragma unroll
            for (int s = 0; s < kSteps; s++) {
                float v[8];
                raw[s].values(v);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    v[i] = n < nrows ? ldexpf(a.scale < 0.0f ? -v[i] : v[i], 14 - ex) : 0.0f;
                    if (s < kSteps - kQLds) {
                        qf[0][s][i] = (_Float16)v[i];
                        if constexpr (kParts == 2) qf[1][s][i] = (_Float16)(v[i] - (float)(_Float16)v[i]);
                    }
                }
                if (s >= kSteps - kQLds)
                    *reinterpret_cast<uint4 *>(s_q + (s - (kSteps - kQLds)) * S::kThreads * 16 + tid * 16) =
                        make_uint4(pack_half(v[0], v[1]), pack_half(v[2], v[3]), pack_half(v[4], v[5]), pack_half(v[6], v[7]));
            }
        }
        floatx16 o[kTiles];
#pragma unroll
        for (int i = 0; i < kTiles; i++) o[i] = floatx16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
        float m = kLow, E = 0.0f, L = 0.0f;

        // staging: item i < 256 holds 4 values of 8 positions of V, the others 32 values of a position of K
        const int P = a.c.page_size, pm = P - 1;
        const int32_t *table = a.s.page_table + b * a.s.table_width;
        uint32_t st[kItems][8];
        float st_ks = 0.0f, st_vs = 0.0f;   // key scale: -1 where the page is not there
        int page[kItems];
        auto item_v = [&](int i) { return S::kWaves == 8 ? wave < 4 : i == 0; };
        // V: position group, first value; K: position, chunk
        auto place_v = [&](int &vg, int &vd) {
            const int it = fresh(tid) & 255;
            vg = it / (D / 4);
            vd = 4 * (it % (D / 4));
        };
        auto place_k = [&](int &kt, int &kc) {
            const int it = fresh(tid) & 255;
            kt = it / (D / 32);
            kc = it % (D / 32);
        };
        auto scaler = [&]() { return (fresh(tid) & 255) % (D / 2) == 0; };  // brings a group's scales
        auto find_page = [&](int tile, int i) {
            int x, y;
            if (item_v(i)) {
                place_v(x, y);
                x = 16 * (x >> 1);
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
                    const int8_t *p = a.c.v + (blk * P + ((tile * T + 16 * (vg >> 1)) & pm) + 4 * (vg & 1)) * D + vd;
#pragma unroll
                    for (int j = 0; j < 8; j++) st[i][j] = *reinterpret_cast<const uint32_t *>(p + ((j & 3) + 8 * (j >> 2)) * D);
                    if (scaler()) {
                        st_ks = ok ? a.c.k_scale[blk] : -1.0f;
                        st_vs = a.c.v_scale[blk];
                    }
                } else {
                    int kt, kc;
                    place_k(kt, kc);
                    const int8_t *p = a.c.k + (blk * P + ((tile * T + kt) & pm)) * D + 16 * kc;
                    const uint4 x = *reinterpret_cast<const uint4 *>(p), y = *reinterpret_cast<const uint4 *>(p + D / 2);
                    st[i][0] = x.x; st[i][1] = x.y; st[i][2] = x.z; st[i][3] = x.w;
                    st[i][4] = y.x; st[i][5] = y.y; st[i][6] = y.z; st[i][7] = y.w;
                }
            }
        };
        auto store = [&](int buf) {
#pragma unroll
            for (int i = 0; i < kItems; i++) {
                if (item_v(i)) {
                    int vg, vd;
                    place_v(vg, vd);
                    char *p = s_v[buf] + L8::v_at(L8::v_row(vd), vg);  // values vd + y: y (D / 4) rows on
                    uint32_t d[8];
#pragma unroll
                    for (int j = 0; j < 8; j++) d[j] = st[i][j] ^ kSign4;
                    *reinterpret_cast<uint4 *>(p) = make_uint4(codes_pair<0>(d[0], d[1]), codes_pair<0>(d[2], d[3]), codes_pair<0>(d[4], d[5]), codes_pair<0>(d[6], d[7]));
                    *reinterpret_cast<uint4 *>(p + L8::v_at(D / 4, 0)) = make_uint4(codes_pair<1>(d[0], d[1]), codes_pair<1>(d[2], d[3]), codes_pair<1>(d[4], d[5]), codes_pair<1>(d[6], d[7]));
                    *reinterpret_cast<uint4 *>(p + L8::v_at(D / 2, 0)) = make_uint4(codes_pair<2>(d[0], d[1]), codes_pair<2>(d[2], d[3]), codes_pair<2>(d[4], d[5]), codes_pair<2>(d[6], d[7]));
                    *reinterpret_cast<uint4 *>(p + L8::v_at(3 * D / 4, 0)) = make_uint4(codes_pair<3>(d[0], d[1]), codes_pair<3>(d[2], d[3]), codes_pair<3>(d[4], d[5]), codes_pair<3>(d[6], d[7]));
                    if (scaler()) {
                        // (the logarithm is the fraction's: it takes a subnormal scale for 0)
                        int e = kZeroExp;
                        const float part = st_vs > 0.0f ? frexpf(st_vs, &e) : 0.0f;
                        s_sc[buf][vg >> 1] = make_float4(st_ks, st_vs, (float)e + __builtin_amdgcn_logf(part), st_ks < 0.0f ? kNoPage : (float)e);
                    }
                } else {
                    int kt, kc;
                    place_k(kt, kc);
                    char *p = s_k[buf] + L8::k_at(kt, 2 * kc);
#pragma unroll
                    for (int x = 0; x < 4; x++)
                        *reinterpret_cast<half8_t *>(p + L8::k_at(0, (x & 1) + (x >> 1) * (D / 16))) = codes_natural(st[i][2 * x], st[i][2 * x + 1]);
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
                float4 sc[kScales];
#pragma unroll
                for (int u = 0; u < kScales; u++) sc[u] = s_sc[buf][step * (kWide / 16) + u * (kSpan / 16)];
                const int ln = fresh(lane);
                const char *kp = s_k[buf] + L8::k_at(kWide * step + (ln & 31), ln >> 5);
                const char *vp = s_v[buf] + L8::v_at(ln & 31, 2 * (kWide / 16) * step + (ln >> 5));
                auto k_frag = [&](int x) {  // step x % kSteps of positions 32 (x / kSteps) ..
                    return *reinterpret_cast<const half8_t *>(kp + L8::k_at(32 * (x / kSteps), 0) + 16 * (x % kSteps));
                };
                auto v_frag = [&](int x) {  // values 32 (x % kTiles) .., positions 16 (x / kTiles) ..
                    return *reinterpret_cast<const half8_t *>(vp + L8::v_at(32 * (x % kTiles), 2 * (x / kTiles)));
                };
                floatx16 s[kSubs];
#pragma unroll
                for (int y = 0; y < kSubs; y++) s[y] = floatx16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
                half8_t kf[kAhead];
#pragma unroll
                for (int x = 0; x < kAhead; x++) kf[x] = k_frag(x);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int x = 0; x < kSubs * kSteps; x++) {
                    const half8_t k = kf[x % kAhead];
                    if (x + kAhead < kSubs * kSteps) kf[x % kAhead] = k_frag(x + kAhead);
                    const int i = x % kSteps, y = x / kSteps;
                    if (i >= kSteps - kQLds) {
                        const half8_t qx = *reinterpret_cast<const half8_t *>(s_q + (i - (kSteps - kQLds)) * S::kThreads * 16 + tid * 16);
                        s[y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, qx, s[y], 0, 0, 0);
                    } else {
#pragma unroll
                        for (int pt = 0; pt < kParts; pt++) s[y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, qf[pt][i < kSteps - kQLds ? i : 0], s[y], 0, 0, 0);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                half8_t vf[kAhead];
#pragma unroll
                for (int x = 0; x < kAhead; x++) vf[x] = v_frag(x);
                __builtin_amdgcn_sched_barrier(0);
                // scores of one page are s[y][kOf v] .. of it: kOf of them in a lane
                float worst = sc[0].w;
#pragma unroll
                for (int u = 1; u < kScales; u++) worst = fmaxf(worst, sc[u].w);
                if (!(p0 >= all_lo && all_hi - p0 >= kWide && worst < kNoPage)) {
                    const int to = hi - p0 - 4 * (ln >> 5), from = a.window ? __builtin_elementwise_sub_sat(to, (int)a.window) : -p0 - kWide;
#pragma unroll
                    for (int j = 0; j < 16 * kSubs; j++) {
                        const int t = 8 * (j >> 2) + (j & 3);
                        const bool see = (t >= from) & (t < to) & (sc[j / kOf].w < kNoPage);
                        s[j >> 4][j & 15] = see ? s[j >> 4][j & 15] : -INFINITY;
                    }
                }
                float f[kScales], top[kScales], e[kScales], mn = m;
#pragma unroll
                for (int u = 0; u < kScales; u++) {
                    float x = s[u * kOf >> 4][u * kOf & 15];
#pragma unroll
                    for (int j = 1; j < kOf; j++) x = fmaxf(x, s[(u * kOf + j) >> 4][(u * kOf + j) & 15]);
                    x = max_xor32(x);
                    // a masked score is -inf whatever the page's scale holds
                    f[u] = fmaxf(fac * sc[u].x, 0x1p-126f);
                    top[u] = ceilf(x * f[u]);
                    e[u] = x == -INFINITY ? (float)kZeroExp : sc[u].w;
                    mn = fmaxf(mn, top[u]);
                }
                const float down = m - mn;
                // E grows by 4 more than it has to, so that it seldom does (8192 tokens of 24 / 4 heads of 256 934 us, 960 by
                // no more); not where the products are wanted to fp32's precision, 2^-25 of the largest then
                float need = (top[0] - mn) + e[0];
#pragma unroll
                for (int u = 1; u < kScales; u++) need = fmaxf(need, (top[u] - mn) + e[u]);
                const float En = need > E + down ? need + (BF16 ? 4.0f : 0.0f) : E + down;
                const float turn = down + (E - En);
                L *= pow2_down(down);
                if (__any(turn < 0.0f)) {
                    const float x = pow2_down(turn);
#pragma unroll
                    for (int i = 0; i < kTiles; i++) o[i] *= x;
                }
                m = mn;
                E = En;
                half8_t pf[2 * kSubs][kParts];  // positions 16 x .. of the step
                auto weights = [&](int u) {     // of page u of the step
                    uint32_t r[kOf / 2];
                    float sum = 0.0f;
                    if constexpr (BF16) {
                        // a page whose values are not seen may hold any scale
                        const float lw = e[u] > (float)kZeroExp ? fmaxf(sc[u].z + ((float)kProbExp - En), -60.0f) : -60.0f;
                        const float c = lw - mn;
#pragma unroll
                        for (int j = 0; j < kOf; j += 2) {
                            const int k = u * kOf + j;
                            const float p0x = __builtin_amdgcn_exp2f(fmaf(s[k >> 4][k & 15], f[u], c));
                            const float p1x = __builtin_amdgcn_exp2f(fmaf(s[k >> 4][(k & 15) + 1], f[u], c));
                            sum += p0x + p1x;
                            r[j / 2] = pack_half(p0x, p1x);   // 2^14 at most, as E is
                        }
                        L = fmaf(sum, __builtin_amdgcn_exp2f(-lw), L);
#pragma unroll
                        for (int x = 0; x < kOf / 8; x++)
                            pf[u * (kOf / 8) + x][0] = __builtin_bit_cast(half8_t, make_uint4(r[4 * x], r[4 * x + 1], r[4 * x + 2], r[4 * x + 3]));
                    } else {
                        float minus = -1.0f;
                        asm("" : "+v"(minus));   // fma takes an fp16 number as it is, a subtraction would widen it first
                        const float w = e[u] > (float)kZeroExp ? fminf(ldexpf(sc[u].y, (int)((float)kProbExp - En)), 0x1p100f) : 0.0f;
#pragma unroll
                        for (int j = 0; j < kOf; j += 2) {
                            const int k = u * kOf + j;
                            const float p0x = __builtin_amdgcn_exp2f(fmaf(s[k >> 4][k & 15], f[u], -mn));
                            const float p1x = __builtin_amdgcn_exp2f(fmaf(s[k >> 4][(k & 15) + 1], f[u], -mn));
                            sum += p0x + p1x;
                            const float x0 = p0x * w, x1 = p1x * w;   // 2^14 at most, as E is
                            uint32_t hw = pack_half(x0, x1);
                            asm("" : "+v"(hw));                      // once: what is taken off is what was kept
                            const half2_t h = __builtin_bit_cast(half2_t, hw);
                            pf[k >> 3][0][k & 7] = h[0];
                            pf[k >> 3][0][(k & 7) + 1] = h[1];
                            pf[k >> 3][kParts - 1][k & 7] = (_Float16)fmaf((float)h[0], minus, x0);
                            pf[k >> 3][kParts - 1][(k & 7) + 1] = (_Float16)fmaf((float)h[1], minus, x1);
                        }
                        L += sum;
                    }
                };
#pragma unroll
                for (int u = 0; u < kScales / kSubs; u++) weights(u);
                __builtin_amdgcn_sched_barrier(kSchedPV);
#pragma unroll
                for (int x = 0; x < 2 * kSubs * kTiles; x++) {
                    if (kSubs == 2 && x == 2 * kTiles) {
#pragma unroll
                        for (int u = kScales / kSubs; u < kScales; u++) weights(u);
                    }
                    const half8_t v = vf[x % kAhead];
                    if (x + kAhead < 2 * kSubs * kTiles) vf[x % kAhead] = v_frag(x + kAhead);
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
                put_shared4(p, S::kRegs * 256 + lane * 16, m, E, L, 0.0f);
            }, [&](unsigned x, unsigned step, unsigned) {
                // of the node's two slots this workgroup holds one; a sum of two does not ask for their order
                if (nrows == 0) return;
                const __amdgpu_buffer_rsrc_t p = slot(held == x ? x + step : x);
                held = x;
                const floatx4 st = get_shared4(p, S::kRegs * 256 + lane * 16);
                constexpr int kAtOnce = S::kRegs / 4 < 16 ? S::kRegs / 4 : 16;  // 16-byte loads in flight
                float qa = 0.0f, qb = 0.0f;
#pragma unroll
                for (int i0 = 0; i0 < S::kRegs / 4; i0 += kAtOnce) {
                    floatx4 v[kAtOnce];
#pragma unroll
                    for (int i = 0; i < kAtOnce; i++) v[i] = get_shared4(p, (i0 + i) * 1024 + lane * 16);
                    __builtin_amdgcn_sched_barrier(0);
                    if (i0 == 0) {
                        const State t = join(State{m, E, L}, State{st[0], st[1], st[2]}, qa, qb);
                        m = t.m;
                        E = t.E;
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
            const float inv = L > 0.0f ? 1.0f / L : 0.0f;
            int64_t token;
            int head;
            row_of(token, head);
            const int64_t off = ((q.first + token) * a.hq + head) * D;
            const int ex = (int)E + kCodeExp - kProbExp;
            // value 4 x + y is in row x + y (D / 4) of O^T; this lane has the rows 32 i + 8 j + 4 hh + c
#pragma unroll
            for (int z = 0; z < D / 8; z++) {
                const int x = (z >> 2) * 8 + (z & 3);   // and + 4 hh
                float v[4];
#pragma unroll
                for (int y = 0; y < 4; y++) {
                    const int row = x + y * (D / 4);
                    v[y] = ldexpf(o[row >> 5][((row & 31) >> 3) * 4 + (row & 3)] * inv, ex);
                }
                const int64_t d = off + 4 * (x + 4 * hh);
                if constexpr (BF16) {
                    uint2 u;
                    u.x = pack_bf16(v[0], v[1]);
                    u.y = pack_bf16(v[2], v[3]);
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.o) + d) = u;
                } else {
                    *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + d) = make_float4(v[0], v[1], v[2], v[3]);
                }
            }
        }
        at = unit1;
    }
}

template <int D, bool BF16>
hipError_t launch_t(const AttnArgs &a, int num_cu, hipStream_t stream) {
    if (a.c.page_size == 16) k_attn_prompt<D, BF16, true><<<num_cu, Shape<D, BF16>::kThreads, 0, stream>>>(a, num_cu);
    else k_attn_prompt<D, BF16, false><<<num_cu, Shape<D, BF16>::kThreads, 0, stream>>>(a, num_cu);
    return hipGetLastError();
}

template <int D>
hipError_t launch_d(const AttnArgs &a, int bf16, int num_cu, hipStream_t stream) {
    return bf16 ? launch_t<D, true>(a, num_cu, stream) : launch_t<D, false>(a, num_cu, stream);
}

}  // namespace

int64_t attn_prompt_bytes(int head_dim, int num_cu) {
    const int64_t regs = head_dim / 2;
    return 4 * 2 * (int64_t)num_cu * 8 * 64 * (regs + 4);
}

hipError_t launch_attn_prompt(const AttnArgs &a, int bf16, int num_cu, hipStream_t stream) {
    switch (a.c.head_dim) {
        case 64: return launch_d<64>(a, bf16, num_cu, stream);
        case 128: return launch_d<128>(a, bf16, num_cu, stream);
        default: return launch_d<256>(a, bf16, num_cu, stream);
    }
}

}  // namespace w4a8
