"""The attention operators on the GPU against their 64-bit forms (tests/attention_ref.py).

Error bounds, u = 2^-24 (fp32), stated before the first run:

rope       sum of squares: D products and additions, at most 16 deep per lane and exchange, its
           mean, sum, root and quotient: 12 u on the factor; two products for the weight; the angle
           in turns is rounded once to fp32 (pi u), sine and cosine are good to 2 ulp and rounded
           by attn_factor; two products and a sum: in all 32 u of |a| + |b|.  bf16 adds
           half a step, 2^-8 of the value.
append     bit-exact.
attention  delta bounds the score's sum of |terms|; its fp32 sum of D products in any order is off
           by at most (D + 4) u delta, scaling and the exponent's argument by 4 u of the score and
           of the maximum each (both at most delta): (D + 16) u delta = e, and exp2 is good to 2 ulp.  A
           weight is off by e + 4 u relatively, their sum too: 2 e + 8 u of A = sum p |v|.  The
           sums over positions add at most one rounding per 32-position step and 32 inside it:
           (L / 32 + 40) u A, for numerator and denominator; joining at most 64 parts adds 70 u A.
           Probabilities as fp16: 2^-11 A (fp32: two fp16 numbers, 2^-21 A), and what is under
           fp16's range is off by at most 2^-25 2^-14 of the row's largest weight (T).  fp32 queries
           as two fp16 numbers: 2^-22 delta on the score.  The output's half step: 2^-8 (bf16)
           or 2^-24 of the value.
"""
import numpy as np
import pytest
import torch

import attention_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from w4a8_codebook_gemm_amd import attention
    attention.lib()
    return attention


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def f32(t):
    return t.detach().to(torch.float32).cpu().numpy()


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(DEV)


# ----------------------------------------------------------------------------- head norm and rotary positions

ROPE = [
    # M, Hq, Hkv, D, R, interleaved, norm, gated, scaling, x, out, first position
    (1, 24, 4, 256, 64, False, True, True, "plain", BF, BF, 262143),
    (1, 1, 1, 64, 16, True, True, False, "plain", F32, F32, 0),
    (3, 5, 1, 64, 48, False, True, False, "linear", F32, F32, 1000),
    (7, 32, 8, 128, 128, True, True, False, "yarn", BF, F32, 100000),
    (7, 32, 8, 128, 128, False, False, False, "ntk", F32, BF, 5),
    (33, 3, 2, 256, 256, False, True, True, "plain", F32, F32, 50000),
    (65, 9, 3, 64, 64, True, False, True, "plain", BF, BF, -70),
    (1025, 6, 2, 128, 80, False, True, True, "yarn", F32, F32, 77),
    (2050, 4, 1, 256, 16, True, True, False, "plain", BF, BF, 3),
    (4099, 2, 2, 64, 32, False, True, False, "plain", F32, BF, 2 ** 31 - 4100),
]


@pytest.mark.parametrize("M,Hq,Hkv,D,rot,inter,norm,gated,scaling,xdt,odt,first", ROPE)
def test_rope(A, M, Hq, Hkv, D, rot, inter, norm, gated, scaling, xdt, odt, first):
    rng = np.random.default_rng(M * 7 + D)
    freq, attn = A.rope_frequencies(rot, 1e6, scaling, 8.0, 4096.0, device=DEV)
    pos = rng.permutation(np.arange(first, first + M)).astype(np.int32)
    w = [(rng.standard_normal(D) * 0.3).astype(np.float32) if norm else None for _ in range(2)]
    x = [dev(rng.standard_normal((M, h, 2 * D if gated else D)).astype(np.float32) * 3, xdt)[:, :, :D] for h in (Hq, Hkv)]
    x[0][0] = 0           # a zero row stays zero
    y = A.qk_norm_rope(x[0], x[1], dev(pos), freq, q_weight=None if w[0] is None else dev(w[0]),
                       k_weight=None if w[1] is None else dev(w[1]), eps=1e-6, weight_offset=1.0 if norm else 0.0,
                       interleaved=inter, attn_factor=attn, out_dtype=odt)
    torch.cuda.synchronize()
    for xi, yi, wi in zip(x, y, w):
        assert yi.dtype == odt and yi.is_contiguous()
        ref, size = R.rope(f64(xi), pos, f64(freq), wi, 1e-6, 1.0, inter, attn)
        err = np.abs(f64(yi) - ref)
        bound = 32 * U * size + half_step(odt) * np.abs(ref)
        assert np.all(err <= bound), float((err / np.maximum(bound, 1e-300)).max())


def test_rope_in_place_queries_only_and_layouts(A):
    freq, _ = A.rope_frequencies(64, device=DEV)
    q = torch.randn(37, 6, 128, device=DEV, dtype=BF)
    w = torch.randn(128, device=DEV)
    pos = torch.arange(37, dtype=torch.int32, device=DEV)
    want, none = A.qk_norm_rope(q, None, pos, freq, q_weight=w)
    assert none is None
    turned = q.transpose(0, 1).contiguous().transpose(0, 1)    # heads outermost in memory
    got, _ = A.qk_norm_rope(turned, None, pos, freq, q_weight=w)
    same = q.clone()
    A.qk_norm_rope(same, None, pos, freq, q_weight=w, out=(same, None))
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(same, want)


# ----------------------------------------------------------------------------- the cache

class Batch:
    """Sequences with pages in random order; new tokens and lengths as given."""

    def __init__(self, A, rng, new, lens, page, extra_width=1, spare=2, rows_behind=0):
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        width = max(need + [1]) + extra_width
        self.table = np.full((len(new), width), 2 ** 30, np.int32)   # entries past a sequence's end are not read
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.lens = np.array(lens, np.int32)
        self.M = int(self.cu[-1]) + rows_behind
        self.A = A

    def seqs(self):
        return self.A.Sequences(dev(self.table), dev(self.cu), dev(self.lens))


def random_cache(A, rng, pages, hkv, page, d, spread=1.0):
    """Codes of every value -127..127 and scales over a range of 30."""
    codes = [rng.integers(-127, 128, (pages, hkv, page, d)).astype(np.int8) for _ in range(2)]
    scales = [(spread * np.exp(rng.uniform(-3.4, 0, (pages, hkv)))).astype(np.float32) / 100 for _ in range(2)]
    return codes, scales, A.KVCache(dev(codes[0]), dev(codes[1]), dev(scales[0]), dev(scales[1]))


APPEND = [
    # new, lens, Hkv, D, page, dtype, magnitude
    ([1], [1], 1, 64, 16, BF, 1.0),
    ([1, 1, 1], [5, 16, 17], 2, 256, 16, F32, 1.0),
    ([1] * 70, list(range(1, 71)), 3, 128, 32, BF, 30.0),
    ([0, 17, 0, 40, 1], [9, 17, 0, 55, 33], 4, 256, 16, BF, 1.0),
    ([100, 1, 257], [100, 64, 300], 2, 64, 64, F32, 1e-3),
    ([513], [600], 1, 256, 256, BF, 2.0),
    ([300, 300], [300, 333], 2, 128, 256, F32, 500.0),
    ([5, 9], [3, 9], 1, 64, 16, F32, 1.0),          # a length shorter than its new tokens
    ([1, 1], [1000, 20], 2, 128, 128, BF, 1e4),      # page past the table's width: held to it
    ([0] * 59 + [200], [7] * 59 + [230], 3, 256, 256, F32, 2.0),  # few tokens a sequence, all of them one's
    ([0] * 149 + [290, 290], [0] * 149 + [290, 320], 1, 128, 256, BF, 2.0),
    ([2] * 130, [2 + i % 40 for i in range(130)], 5, 64, 64, BF, 1.0),
]


@pytest.mark.parametrize("new,lens,Hkv,D,page,dtype,mag", APPEND)
def test_append(A, new, lens, Hkv, D, page, dtype, mag):
    rng = np.random.default_rng(sum(new) + D)
    b = Batch(A, rng, new, lens, page, rows_behind=3)
    codes, scales, cache = random_cache(A, rng, b.pages, Hkv, page, D, 10.0)
    scales[0][:, 0] = 0                       # a head whose pages hold zeros so far
    codes[0][:, 0] = 0
    cache.k.copy_(dev(codes[0]))
    cache.k_scale.copy_(dev(scales[0]))
    x = [dev((rng.standard_normal((b.M, 2 * Hkv, D)) * mag).astype(np.float32), dtype)[:, i * Hkv:(i + 1) * Hkv] for i in (0, 1)]
    x[1][0] = 0
    seqs = b.seqs()
    for _ in range(2):                        # the second call finds its own tokens' scales: nothing changes
        A.kv_append(x[0], x[1], cache, seqs)
    torch.cuda.synchronize()
    for xi, c, s, got_c, got_s in zip(x, codes, scales, (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
        R.append(f32(xi), c, s, b.table, b.cu, b.lens, b.pages)
        assert np.array_equal(got_s.cpu().numpy().view(np.uint32), s.view(np.uint32))
        assert np.array_equal(got_c.cpu().numpy(), c)


def test_append_token_by_token(A):
    """A page filled one token at a time with growing values: the codes stay within one step of the
    final scale, and the steps are the definition's."""
    rng = np.random.default_rng(5)
    P, H, D = 64, 2, 128
    cache = A.KVCache.empty(2, H, P, D, device=DEV)
    codes, scales = np.zeros((2, H, P, D), np.int8), np.zeros((2, H), np.float32)
    xs = (rng.standard_normal((P + 9, H, D)) * 1.1 ** np.arange(P + 9)[:, None, None]).astype(np.float32)
    table = np.array([[1, 0]], np.int32)
    for t in range(P + 9):
        s = A.Sequences(dev(table), dev(np.array([0, 1], np.int32)), dev(np.array([t + 1], np.int32)))
        A.kv_append(dev(xs[t:t + 1]), dev(xs[t:t + 1]), cache, s)
        R.append(xs[t:t + 1], codes, scales, table, np.array([0, 1]), np.array([t + 1]), 2)
    torch.cuda.synchronize()
    assert np.array_equal(cache.k.cpu().numpy(), codes) and np.array_equal(cache.v_scale.cpu().numpy(), scales)
    held = codes[1].astype(np.float64) * scales[1][:, None, None]
    assert np.all(np.abs(held - xs[:P].transpose(1, 0, 2)) <= scales[1][:, None, None] * (1 + 1e-6))


def test_append_extremes(A):
    """Zeros, the smallest and largest finite numbers."""
    P, H, D = 16, 1, 64
    for mags in ([0.0, 0.0], [1e-45, 1e-44], [1e-38, 3.3e38], [3.4e38, 1e-45], [0.0, 1e-41]):
        cache = A.KVCache.empty(1, H, P, D, device=DEV)
        codes, scales = np.zeros((1, H, P, D), np.int8), np.zeros((1, H), np.float32)
        for t, m in enumerate(mags):
            x = (np.linspace(-1, 1, D).reshape(1, 1, D) * m).astype(np.float32)
            s = A.Sequences(dev(np.zeros((1, 1), np.int32)), dev(np.array([0, 1], np.int32)), dev(np.array([t + 1], np.int32)))
            A.kv_append(dev(x), dev(x), cache, s)
            R.append(x, codes, scales, np.zeros((1, 1), np.int32), np.array([0, 1]), np.array([t + 1]), 1)
        torch.cuda.synchronize()
        assert np.array_equal(cache.k_scale.cpu().numpy(), scales), mags
        assert np.array_equal(cache.k.cpu().numpy(), codes), mags


# ----------------------------------------------------------------------------- attention

def check_attention(A, q, b, codes, scales, cache, causal=True, window=0, workspace=None, scale=None, run=None):
    d = q.shape[-1]
    sm = d ** -0.5 if scale is None else scale
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    if run is None:
        A.kv_attention(q, cache, b.seqs(), scale=sm, causal=causal, window=window, workspace=workspace, out=out)
    else:
        out = run(out)
    torch.cuda.synchronize()
    ref, size, top, delta = R.attention(f64(q), codes[0], scales[0], codes[1], scales[1], b.table, b.cu, b.lens, sm, causal, window)
    got = f64(out)
    behind = np.isnan(ref)
    assert np.all(got[behind] == 7.0)                     # rows of no sequence
    ref = np.where(behind, 7.0, ref)
    wide = q.dtype == F32
    length = int(max(b.lens.max(), 1))
    e = ((d + 16) * U + (2.0 ** -22 if wide else 0)) * delta
    bound = (2 * e + 8 * U + 2 * (length / 32 + 40) * U + 70 * U + (2.0 ** -21 if wide else 2.0 ** -11)) * size
    bound = bound + 2.0 ** -39 * top + half_step(q.dtype) * (np.abs(ref) + bound)
    err = np.abs(got - ref)
    assert np.all(err <= bound), float((err / np.maximum(bound, 1e-300)).max())


ATTN = [
    # new, lens, Hq, Hkv, D, page, dtype, causal, window
    ([1], [1], 1, 1, 64, 16, BF, True, 0),
    ([1], [777], 24, 4, 256, 16, BF, True, 0),
    ([1, 1, 1], [33, 1, 64], 6, 2, 128, 32, F32, True, 0),
    ([1] * 9, [5, 700, 64, 65, 1, 1023, 128, 31, 32], 8, 1, 128, 64, BF, True, 0),
    ([1, 1], [4100, 37], 12, 2, 256, 128, F32, True, 0),
    ([0, 1, 0, 3, 0], [20, 40, 0, 70, 1], 4, 4, 64, 16, BF, True, 0),
    ([4, 2, 5], [400, 90, 5], 16, 2, 256, 32, F32, True, 0),
    ([7], [300], 20, 5, 128, 64, BF, True, 100),
    ([1, 1], [500, 9], 10, 2, 64, 16, F32, True, 17),
    ([1, 2], [500, 90], 32, 1, 128, 256, BF, False, 0),
    ([33], [33], 7, 1, 64, 16, F32, True, 0),
    ([130, 65, 1], [130, 200, 50], 6, 2, 128, 32, BF, True, 0),
    ([200], [517], 12, 2, 256, 64, BF, True, 0),
    ([100, 3], [150, 300], 4, 2, 256, 16, F32, True, 0),
    ([257, 64], [257, 64], 4, 4, 64, 64, BF, True, 50),
    ([150], [400], 8, 2, 128, 128, F32, True, 1),
    ([90, 120], [90, 333], 3, 1, 128, 32, F32, False, 0),
    ([10, 300], [4, 290], 2, 1, 64, 16, BF, True, 0),       # first rows stand in front of position 0
    ([70], [700], 5, 1, 256, 256, BF, True, 200),
]


@pytest.mark.parametrize("new,lens,Hq,Hkv,D,page,dtype,causal,window", ATTN)
def test_attention(A, new, lens, Hq, Hkv, D, page, dtype, causal, window):
    rng = np.random.default_rng(sum(lens) + D)
    b = Batch(A, rng, new, lens, page, rows_behind=2)
    codes, scales, cache = random_cache(A, rng, b.pages, Hkv, page, D)
    q = dev(rng.standard_normal((b.M, 2 * Hq, D)).astype(np.float32) * 2, dtype)[:, Hq:]
    check_attention(A, q, b, codes, scales, cache, causal, window)


@pytest.mark.parametrize("new,lo,hi,count,Hq,Hkv,D,dtype", [
    (1, 500, 6000, 40, 24, 4, 256, BF),       # several units and parts of units for a workgroup, blocks of 16 rows
    (1, 20, 1500, 300, 8, 8, 64, F32),        # more sequences than a wave has lanes
    (7, 300, 2500, 40, 12, 3, 128, BF),       # blocks of 32 rows
    (60, 60, 1200, 70, 8, 2, 128, BF),        # many rows, more sequences than lanes
    (90, 90, 900, 10, 8, 2, 256, F32),
])
def test_attention_of_many_units(A, new, lo, hi, count, Hq, Hkv, D, dtype):
    """Batches large enough that a workgroup has several units, cut anywhere."""
    rng = np.random.default_rng(D + count)
    lens = rng.integers(lo, hi, count)
    b = Batch(A, rng, [new] * count, list(lens), 16)
    codes, scales, cache = random_cache(A, rng, b.pages, Hkv, 16, D)
    q = dev(rng.standard_normal((b.M, Hq, D)).astype(np.float32), dtype)
    check_attention(A, q, b, codes, scales, cache)


@pytest.mark.parametrize("count,lo,hi,Hq,Hkv,D,page,dtype,window", [
    (300, 1, 60, 16, 8, 64, 16, BF, 0),            # a unit or more for each wave
    (300, 30, 260, 24, 8, 128, 32, F32, 0),
    (700, 1, 150, 20, 5, 128, 16, BF, 0),
    (280, 100, 300, 8, 8, 64, 64, F32, 70),
    (150, 40, 90, 32, 16, 128, 16, BF, 33),
])
@pytest.mark.parametrize("shape", ["alike", "some empty", "one long", "several tokens"])
def test_attention_of_many_short_sequences(A, count, lo, hi, Hq, Hkv, D, page, dtype, window, shape):
    """Batches with a unit or more for each wave, and those that the same launch must share out differently."""
    rng = np.random.default_rng(count + D)
    new, lens = [1] * count, [int(x) for x in rng.integers(lo, hi, count)]
    if shape == "some empty":
        new = [int(x) for x in rng.integers(0, 2, count)]
    elif shape == "one long":
        lens[count // 3] = 9000
    elif shape == "several tokens":
        new = [min(int(x), 16 * Hkv // Hq) for x in rng.integers(1, 4, count)]
    b = Batch(A, rng, new, lens, page, rows_behind=3)
    codes, scales, cache = random_cache(A, rng, b.pages, Hkv, page, D)
    b.table[5, 0] = -1
    b.table[7] = -1
    q = dev(rng.standard_normal((b.M, Hq, D)).astype(np.float32), dtype)
    check_attention(A, q, b, codes, scales, cache, window=window)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("new", [[1, 1, 1], [40, 90, 20]])
def test_attention_pages_given_up(A, dtype, new):
    """Pages marked -1, past the cache, or all of a sequence's."""
    rng = np.random.default_rng(3)
    b = Batch(A, rng, new, [200, 300, 90], 16)
    b.table[0, 2] = -1
    b.table[0, 5:8] = 2 ** 31 - 1
    b.table[1, 0] = b.pages
    b.table[2, :6] = -1
    codes, scales, cache = random_cache(A, rng, b.pages, 2, 16, 128)
    q = dev(rng.standard_normal((b.M, 6, 128)).astype(np.float32), dtype)
    check_attention(A, q, b, codes, scales, cache)
    check_attention(A, q, b, codes, scales, cache, window=40)
    x = dev(rng.standard_normal((b.M, 2, 128)).astype(np.float32), dtype)
    A.kv_append(x, x, cache, b.seqs())
    torch.cuda.synchronize()
    for c, s, gc, gs in zip(codes, scales, (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
        R.append(f32(x), c, s, b.table, b.cu, b.lens, b.pages)
        assert np.array_equal(gc.cpu().numpy(), c) and np.array_equal(gs.cpu().numpy(), s)


def test_offsets_and_lengths_out_of_range(A):
    """Offsets and lengths that a broken program could leave: held to their range."""
    rng = np.random.default_rng(4)
    codes, scales, cache = random_cache(A, rng, 8, 1, 16, 64)
    b = Batch(A, rng, [3, 3], [20, 30], 16, extra_width=0, spare=4)
    b.table[0, 1:] = [7]
    b.lens[1] = 10 ** 6                 # held to the table's width
    q = dev(rng.standard_normal((6, 2, 64)).astype(np.float32))
    check_attention(A, q, b, codes, scales, cache)
    bad = A.Sequences(dev(b.table), dev(np.array([-5, 4, 2 ** 31 - 1], np.int32)), dev(np.array([-3, 2 ** 31 - 1], np.int32)))
    out = A.kv_attention(q, cache, bad)
    A.kv_append(q[:, :1].contiguous(), q[:, 1:].contiguous(), cache, bad)
    torch.cuda.synchronize()
    assert torch.equal(out[:4], torch.zeros_like(out[:4]))


@pytest.mark.parametrize("new,lens", [([1, 1], [300, 40]), ([60, 9], [200, 70])])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_extreme_scales(A, new, lens, dtype):
    """Pages whose values are of quite different sizes, pages of zeros, sharp and flat softmaxes."""
    rng = np.random.default_rng(9)
    D = 128
    for exps, qs in ((np.arange(-20, 20), 4.0), (np.full(40, -100), 0.0), (np.full(40, 90), 1.0), (np.arange(-60, 100, 4), 40.0)):
        b = Batch(A, rng, new, lens, 16)
        codes, scales, cache = random_cache(A, rng, b.pages, 1, 16, D)
        scales[1][:] = 2.0 ** exps[np.arange(b.pages) % len(exps)][:, None]
        scales[1][::7] = 0
        codes[1][::7] = 0
        cache.v.copy_(dev(codes[1]))
        cache.v_scale.copy_(dev(scales[1]))
        q = dev(rng.standard_normal((b.M, 2, D)).astype(np.float32) * qs, dtype)
        check_attention(A, q, b, codes, scales, cache)
        check_attention(A, q, b, codes, scales, cache, scale=-0.02)


@pytest.mark.parametrize("new,lens,D,page,window", [
    ([3, 1], [130, 40], 128, 16, 0),
    ([3, 1], [130, 140], 256, 32, 20),
    ([20, 1], [200, 60], 64, 16, 30),
    ([90, 40], [290, 60], 128, 16, 0),
    ([90, 40], [290, 60], 128, 32, 50),
    ([70, 80], [400, 80], 256, 16, 33),
    ([300, 2], [300, 9], 64, 64, 0),
])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_of_what_is_not_seen(A, new, lens, D, page, window, dtype):
    """Pages that a row does not see may hold any scale, and other rows' queries may be anything: its bits stay."""
    rng = np.random.default_rng(D + window)
    b = Batch(A, rng, new, lens, page)
    _, scales, cache = random_cache(A, rng, b.pages, 2, page, D)
    q = dev(rng.standard_normal((b.M, 6, D)).astype(np.float32), dtype)
    seqs = b.seqs()
    want = A.kv_attention(q, cache, seqs, window=window)
    pos = np.concatenate([np.arange(n - m, n) for m, n in zip(new, lens)])
    seq = np.repeat(np.arange(len(new)), new)
    assert bool(torch.isfinite(want).all())
    for bad in (np.nan, np.inf, -np.inf, -1.0):
        for s in range(len(new)):
            for j in sorted({0, (lens[s] - 1) // page, (lens[s] - new[s]) // page}):
                for side in (cache.k_scale, cache.v_scale):
                    side[b.table[s, j]] = bad
                sees = (seq == s) & (pos >= j * page) & ((pos - window + 1 < (j + 1) * page) | (window == 0))
                got = A.kv_attention(q, cache, seqs, window=window)
                cache.k_scale.copy_(dev(scales[0]))
                cache.v_scale.copy_(dev(scales[1]))
                assert torch.equal(got[dev(~sees)], want[dev(~sees)]), (bad, s, j)
        x = q.clone()
        x[::3, 1] = bad
        got = A.kv_attention(x, cache, seqs, window=window)
        rest = torch.ones(q.shape[:2], dtype=torch.bool, device=DEV)
        rest[::3, 1] = False
        assert torch.equal(got[rest], want[rest]), bad


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (256, 256)])
def test_append_of_values_that_are_not_finite(A, dtype, D, page):
    """They spoil their own page and head, until its first slot is written again."""
    rng = np.random.default_rng(D)
    b = Batch(A, rng, [20, 40, 1], [30, 40, 5], page)
    x = rng.standard_normal((b.M, 2, D)).astype(np.float32)
    caches = []
    for bad in (None, np.nan, np.inf):
        cache = A.KVCache.empty(b.pages, 2, page, D, device=DEV)
        y = x.copy()
        if bad is not None:
            y[19, 1, 5] = bad                     # sequence 0's last token, head 1
        A.kv_append(dev(y, dtype), dev(x, dtype), cache, b.seqs())
        caches.append(cache)
    hit = (b.table[0, 29 // page], 1)
    keep = torch.ones(b.pages, 2, dtype=torch.bool, device=DEV)
    keep[hit] = False
    for c in caches[1:]:
        assert torch.equal(c.v, caches[0].v) and torch.equal(c.v_scale, caches[0].v_scale)
        assert torch.equal(c.k[keep], caches[0].k[keep]) and torch.equal(c.k_scale[keep], caches[0].k_scale[keep])
    again = b.seqs()
    again.seq_lens[0] = 20                        # from position 0 again
    page0 = b.table[0, 0]
    for c in caches:
        A.kv_append(dev(x, dtype), dev(x, dtype), c, again)
    for c in caches[1:]:
        assert torch.equal(c.k_scale[page0], caches[0].k_scale[page0])
        assert torch.equal(c.k[page0, :, :min(20, page)], caches[0].k[page0, :, :min(20, page)])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_query_magnitudes(A, dtype):
    """Queries from 2^-100 to 2^60 within a row and between rows."""
    rng = np.random.default_rng(10)
    b = Batch(A, rng, [1, 30], [100, 90], 16)
    codes, scales, cache = random_cache(A, rng, b.pages, 2, 16, 64)
    q = rng.standard_normal((b.M, 4, 64))
    q[0] *= 2.0 ** rng.integers(-40, 0, (4, 64))
    q[1] *= 2.0 ** -100
    q[2] *= 2.0 ** 60
    q[3] = 0
    check_attention(A, dev(q.astype(np.float32), dtype), b, codes, scales, cache, scale=0.3)


def test_attention_long_offsets(A):
    """A cache over 2^32 bytes: its last pages are read and written."""
    pages, H, P, D = 70000, 1, 256, 256
    cache = A.KVCache(*[torch.zeros((pages, H, P, D), dtype=torch.int8, device=DEV) for _ in range(2)],
                      *[torch.ones((pages, H), device=DEV) for _ in range(2)])
    rng = np.random.default_rng(11)
    x = dev(rng.standard_normal((300, H, D)).astype(np.float32))
    s = A.Sequences(dev(np.array([[pages - 1, pages - 3]], np.int32)), dev(np.array([0, 300], np.int32)), dev(np.array([300], np.int32)))
    small = A.KVCache.empty(4, H, P, D, device=DEV)
    t = A.Sequences(dev(np.array([[3, 1]], np.int32)), dev(np.array([0, 300], np.int32)), dev(np.array([300], np.int32)))
    A.kv_append(x, x, cache, s)
    A.kv_append(x, x, small, t)
    q = dev(rng.standard_normal((300, 2, D)).astype(np.float32))
    assert torch.equal(A.kv_attention(q, cache, s), A.kv_attention(q, small, t))
    assert torch.equal(cache.k[pages - 1], small.k[3]) and torch.equal(cache.v[pages - 3, 0, :44], small.v[1, 0, :44])
    assert int(cache.k[:pages - 3].abs().max()) == 0


@pytest.mark.parametrize("new,dtype", [([1, 1, 1, 1], BF), ([1, 3, 1, 2], F32), ([300, 20, 150, 1], BF)])
def test_attention_is_deterministic_and_leaves_its_workspace(A, new, dtype):
    rng = np.random.default_rng(12)
    b = Batch(A, rng, new, [3000, 700, 2000, 1500], 32)
    codes, scales, cache = random_cache(A, rng, b.pages, 2, 32, 128)
    q = dev(rng.standard_normal((b.M, 12, 128)).astype(np.float32), dtype)
    ws = A.kv_attention_workspace(b.M, 4, 12, 2, 128, DEV)
    seqs = b.seqs()
    first = A.kv_attention(q, cache, seqs, workspace=ws)
    for _ in range(5):
        assert torch.equal(A.kv_attention(q, cache, seqs, workspace=ws), first)
    assert torch.equal(A.kv_attention(q, cache, seqs), first)
    # the same workspace for another shape in between
    small = Batch(A, rng, [2], [50], 32)
    check_attention(A, q[:2], small, codes, scales, cache, workspace=ws)
    assert torch.equal(A.kv_attention(q, cache, seqs, workspace=ws), first)


def test_sequences_that_share_pages(A):
    """A prefix in the tables of several sequences, and a page at two places of one."""
    rng = np.random.default_rng(15)
    for new in ([1, 1, 3], [30, 60, 45]):
        b = Batch(A, rng, new, [100, 90, 150], 16)
        b.table[1, :5] = b.table[0, :5]
        b.table[2, :3] = b.table[0, 2:5]
        b.table[2, 7] = b.table[2, 4]
        codes, scales, cache = random_cache(A, rng, b.pages, 2, 16, 128)
        q = dev(rng.standard_normal((b.M, 8, 128)).astype(np.float32), BF)
        check_attention(A, q, b, codes, scales, cache)


@pytest.mark.parametrize("M,B", [(1, 3), (500, 2), (300, 400)])
def test_batches_without_a_token_or_a_length(A, M, B):
    """Rows that belong to no sequence, and rows whose sequences have length zero."""
    rng = np.random.default_rng(17)
    codes, scales, cache = random_cache(A, rng, 4, 8, 16, 64)
    zeros = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    table = torch.zeros(B, 2, dtype=torch.int32, device=DEV)
    q = torch.randn(M, 8, 64, device=DEV)
    out = torch.full_like(q, 5.0)
    none = A.Sequences(table, zeros, torch.full((B,), 20, dtype=torch.int32, device=DEV))
    A.kv_attention(q, cache, none, out=out)
    A.kv_append(q, q, cache, none)
    assert bool((out == 5.0).all())
    cu = torch.clamp(torch.arange(B + 1, device=DEV) * (-(-M // B)), max=M).to(torch.int32)
    empty = A.Sequences(table, cu, zeros[:B].clone())
    A.kv_attention(q, cache, empty, out=out)
    A.kv_append(q, q, cache, empty)
    assert bool((out == 0).all())
    assert np.array_equal(cache.k.cpu().numpy(), codes[0]) and np.array_equal(cache.v_scale.cpu().numpy(), scales[1])


def test_two_graphs_that_share_a_workspace(A):
    """Captured calls of quite different shapes on one workspace, replayed in turn with eager calls between."""
    rng = np.random.default_rng(16)
    codes, scales, cache = random_cache(A, rng, 400, 2, 32, 128)
    ws = A.kv_attention_workspace(512, 4, 12, 2, 128, DEV)
    runs = []
    for new, lens, dtype in (([1, 1, 1], [3000, 700, 2100], BF), ([300, 40], [1500, 900], BF), ([4, 2], [2500, 30], F32)):
        b = Batch(A, rng, new, lens, 32)
        b.table = rng.integers(0, 400, b.table.shape).astype(np.int32)
        q, seqs = dev(rng.standard_normal((b.M, 12, 128)).astype(np.float32), dtype), b.seqs()
        runs.append((q, seqs, A.kv_attention(q, cache, seqs), torch.empty_like(q)))
    torch.cuda.synchronize()
    graphs = []
    for q, seqs, _, out in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            A.kv_attention(q, cache, seqs, workspace=ws, out=out)
        graphs.append(g)
    for turn in range(6):
        for i in rng.permutation(len(runs)):
            runs[i][3].fill_(3.0)
            graphs[i].replay()
            if turn % 2:
                q, seqs, want, _ = runs[(i + 1) % len(runs)]
                assert torch.equal(A.kv_attention(q, cache, seqs, workspace=ws), want)
            assert torch.equal(runs[i][3], runs[i][2])


def test_streams_and_two_calls_at_once(A):
    """Calls on other streams than the default, with a workspace each, at the same time."""
    rng = np.random.default_rng(13)
    b = Batch(A, rng, [1, 1], [5000, 3000], 64)
    codes, scales, cache = random_cache(A, rng, b.pages, 2, 64, 256)
    seqs = b.seqs()
    qs = [dev(rng.standard_normal((2, 12, 256)).astype(np.float32), BF) for _ in range(2)]
    want = [A.kv_attention(q, cache, seqs) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = []
    for q, st in zip(qs, streams):
        with torch.cuda.stream(st):
            ws = A.kv_attention_workspace(2, 2, 12, 2, 256, DEV)
            got.append([A.kv_attention(q, cache, seqs, workspace=ws) for _ in range(4)])
    torch.cuda.synchronize()
    for outs, w in zip(got, want):
        assert all(torch.equal(o, w) for o in outs)


def test_layer_captured_and_replayed(A):
    """The whole run as a layer uses it -- quantised projections, norm and rotation, append,
    attention, output projection -- captured once and replayed token by token, against
    the same calls made eagerly and the 64-bit attention."""
    import w4a8_codebook_gemm_amd as w
    torch.manual_seed(0)
    K, Hq, Hkv, D, P, B = 512, 4, 2, 128, 16, 3
    quant = lambda n, k, s: w.quantize_weight(torch.randn(n, k, device=DEV) / k ** 0.5, seed=s)  # noqa: E731
    wq, wk, wv, wo = quant(Hq * D, K, 1), quant(Hkv * D, K, 2), quant(Hkv * D, K, 3), quant(K, Hq * D, 4)
    freq, attn = A.rope_frequencies(64, 1e6, device=DEV)
    nw = torch.randn(D, device=DEV) * 0.1
    lens0 = torch.tensor([15, 40, 0], dtype=torch.int32, device=DEV)
    table = torch.randperm(B * 5, device=DEV).to(torch.int32).view(B, 5)
    cu = torch.arange(B + 1, dtype=torch.int32, device=DEV)

    class Run:
        def __init__(self):
            g = torch.Generator(device=DEV).manual_seed(3)
            self.cache = A.KVCache.empty(B * 5, Hkv, P, D, device=DEV)
            for t in (self.cache.k, self.cache.v):
                t.copy_(torch.randint(-127, 128, t.shape, generator=g, device=DEV, dtype=torch.int32).to(torch.int8))
            self.cache.k_scale.fill_(0.01)
            self.cache.v_scale.fill_(0.02)
            self.lens = lens0.clone()
            self.seqs = A.Sequences(table, cu, self.lens)
            self.x = torch.zeros(B, K, device=DEV)
            self.ws = A.kv_attention_workspace(B, B, Hq, Hkv, D, DEV)

        def step(self):
            self.lens += 1
            q, k, v = w.forward_multi(self.x, [wq, wk, wv])
            q, k = A.qk_norm_rope(q.view(B, Hq, D), k.view(B, Hkv, D), self.lens - 1, freq, q_weight=nw, k_weight=nw,
                                  weight_offset=1.0, attn_factor=attn, out_dtype=F32)
            A.kv_append(k, v.view(B, Hkv, D), self.cache, self.seqs)
            o = A.kv_attention(q, self.cache, self.seqs, workspace=self.ws)
            return q, o, w.forward(o.view(B, Hq * D), wo)

    eager, cap = Run(), Run()
    xs = [torch.randn(B, K, device=DEV) for _ in range(20)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm = Run()
        warm.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = cap.step()
    for i, x in enumerate(xs):
        eager.x.copy_(x)
        cap.x.copy_(x)
        want = eager.step()
        graph.replay()
        if i % 3 == 0:
            torch.cuda.synchronize()
        for a, c in zip(want, got):
            assert torch.equal(a, c), i
        assert torch.equal(eager.cache.k, cap.cache.k) and torch.equal(eager.cache.v_scale, cap.cache.v_scale)
    b = Batch.__new__(Batch)
    b.A, b.table, b.cu, b.lens = A, table.cpu().numpy(), cu.cpu().numpy(), eager.lens.cpu().numpy()
    check_attention(A, want[0], b, [eager.cache.k.cpu().numpy(), eager.cache.v.cpu().numpy()],
                    [eager.cache.k_scale.cpu().numpy(), eager.cache.v_scale.cpu().numpy()], eager.cache)


def test_binding_refusals_on_the_gpu(A):
    rng = np.random.default_rng(14)
    codes, scales, cache = random_cache(A, rng, 4, 2, 16, 64)
    s = A.Sequences(dev(np.zeros((1, 2), np.int32)), dev(np.array([0, 2], np.int32)), dev(np.array([2], np.int32)))
    q = torch.randn(2, 4, 64, device=DEV)
    for bad in (q.half(), q.double()):
        with pytest.raises(TypeError):
            A.kv_attention(bad, cache, s)
    with pytest.raises(ValueError):
        A.kv_attention(q.cpu(), cache, s)
    with pytest.raises(ValueError):
        A.kv_attention(q[:, :, :32], cache, s)
    with pytest.raises(ValueError):
        A.kv_attention(q.transpose(0, 1), cache, s)
    with pytest.raises(ValueError):
        A.kv_attention(q, cache, s, out=torch.empty(2, 4, 32, device=DEV))
    with pytest.raises(A.AttentionError):
        A.kv_attention(q[:, :3].contiguous(), cache, s)
    with pytest.raises(A.AttentionError):
        A.kv_attention(q, cache, s, window=3, causal=False)
    k = torch.randn(2, 2, 64, device=DEV)
    with pytest.raises(TypeError):
        A.kv_append(k, k.bfloat16(), cache, s)
    with pytest.raises(ValueError):
        A.kv_append(k, k[:1], cache, s)
    with pytest.raises(ValueError):
        A.kv_append(k[:, :1], k, cache, s)
    with pytest.raises(ValueError):
        A.KVCache(cache.k, cache.v, cache.k_scale.t(), cache.v_scale)
    with pytest.raises(TypeError):
        A.Sequences(s.page_table.long(), s.cu_tokens, s.seq_lens)
    freq, _ = A.rope_frequencies(32, device=DEV)
    pos = torch.zeros(2, dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError):
        A.qk_norm_rope(q, None, pos.long(), freq)
    with pytest.raises(TypeError):
        A.qk_norm_rope(q, None, pos, freq.float())
    with pytest.raises(ValueError):
        A.qk_norm_rope(q, None, pos[:1], freq)
    with pytest.raises(A.AttentionError):
        A.qk_norm_rope(q, None, pos, torch.zeros(3, dtype=torch.float64, device=DEV))
