"""The attention operators at the ends of the ranges that include/w4a8_attn.h accepts: tokens in front of
position 0, lengths up to 2^31, scales and values at both ends of fp32.  Bounds are those of
tests/test_gpu_attention.py where a test states no other."""
import numpy as np
import pytest
import torch

import attention_ref as R
import test_gpu_attention as T
from test_gpu_attention import A, BF, DEV, F32, Batch, dev, f64, random_cache  # noqa: F401  (A is a fixture)

pytestmark = pytest.mark.gpu
plain_attention = R.attention


def attention_in_front(q, kc, ks, vc, vs, table, cu, lens, scale, causal, window):
    """attention_ref.attention where a token in front of position 0 sees nothing in calls without a causal mask either."""
    o, size, top, delta = plain_attention(q, kc, ks, vc, vs, table, cu, lens, scale, causal, window)
    for b in range(len(lens)):
        n = int(cu[b + 1] - cu[b])
        front = slice(int(cu[b]), int(cu[b]) + max(0, n - max(int(lens[b]), 0)))
        for x in (o, size, top, delta):
            x[front] = 0
    return o, size, top, delta


@pytest.mark.parametrize("new,lens,Hq,Hkv,D,page", [
    ([7], [3], 2, 2, 64, 16),                     # blocks of 16 rows
    ([3, 1, 5], [0, 40, 4], 12, 3, 128, 32),
    ([9, 9], [4, 9], 8, 2, 256, 16),              # blocks of 32 rows
    ([40, 30], [11, 300], 8, 1, 128, 16),         # the prompt kernel
    ([300, 20], [290, 2], 2, 2, 64, 64),
    ([100], [70], 6, 1, 256, 128),
])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("causal", [False, True])
def test_tokens_in_front_of_position_0_see_nothing(A, monkeypatch, new, lens, Hq, Hkv, D, page, dtype, causal):
    rng = np.random.default_rng(sum(new) + D)
    b = Batch(A, rng, new, lens, page, rows_behind=2)
    codes, scales, cache = random_cache(A, rng, b.pages, Hkv, page, D)
    q = dev(rng.standard_normal((b.M, Hq, D)).astype(np.float32), dtype)
    monkeypatch.setattr(R, "attention", attention_in_front)
    T.check_attention(A, q, b, codes, scales, cache, causal=causal)


class Far:
    """One sequence whose length is just below 2^31, nearly all of its pages given up, and the same sequence with
    `cut` positions (a multiple of every tile) taken from its front, where the operators must do the same."""

    def __init__(self, A, rng, new, page, hkv, d, held):
        self.width = 2 ** 31 // page - 1
        self.length = self.width * page - 1        # the last slot of the last page stays free
        self.cut = 2 ** 31 - 4096
        self.pages = held + 2
        far = torch.full((1, self.width), -1, dtype=torch.int32, device=DEV)
        far[0, -held:] = dev(rng.permutation(self.pages)[:held].astype(np.int32))
        near = far[:, self.cut // page:].contiguous()
        self.cu = dev(np.array([0, new], np.int32))
        self.seqs = [A.Sequences(t, self.cu, dev(np.array([n], np.int32)))
                     for t, n in ((far, self.length), (near, self.length - self.cut))]
        _, _, self.cache = random_cache(A, rng, self.pages, hkv, page, d)


@pytest.mark.parametrize("new,Hq,Hkv,D", [
    (1, 6, 1, 256), (1, 8, 2, 128), (1, 2, 2, 64),        # blocks of 16 rows
    (6, 8, 1, 128), (9, 4, 2, 256),                       # blocks of 32 rows
    (100, 2, 1, 256), (90, 4, 2, 128), (300, 3, 1, 64),   # the prompt kernel
])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [1, 500, 1500])
def test_lengths_up_to_2_31_with_a_window(A, new, Hq, Hkv, D, dtype, window):
    """Tile counts and a tile's end pass 2^31 in signed arithmetic: the same bits as 2^31 - 4096 positions earlier."""
    rng = np.random.default_rng(new + D)
    f = Far(A, rng, new, 16, Hkv, D, held=100)
    q = dev(rng.standard_normal((new, Hq, D)).astype(np.float32), dtype)
    far, near = (A.kv_attention(q, f.cache, s, window=window) for s in f.seqs)
    assert bool((near.abs().amax(-1) > 0).all()) and torch.equal(far, near)
    x = dev(rng.standard_normal((new, Hkv, D)).astype(np.float32), dtype)
    caches = [A.KVCache(*(t.clone() for t in (f.cache.k, f.cache.v, f.cache.k_scale, f.cache.v_scale))) for _ in f.seqs]
    for c, s in zip(caches, f.seqs):
        A.kv_append(x, x, c, s)
    assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v_scale, caches[1].v_scale)
    assert not torch.equal(caches[0].k, f.cache.k)


@pytest.mark.parametrize("new,Hq", [(1, 4), (9, 4), (80, 4)])
@pytest.mark.parametrize("page,causal,window", [(16, True, 0), (64, True, 0), (16, False, 0), (16, True, 2 ** 31 - 2)])
def test_lengths_up_to_2_31_without_a_window(A, new, Hq, page, causal, window):
    """All 2^31 positions are walked.  The pages that are there lie in the last tile, so the sums are the same."""
    rng = np.random.default_rng(new)
    f = Far(A, rng, new, page, 1, 64, held=64 // page)
    q = dev(rng.standard_normal((new, Hq, 64)).astype(np.float32), F32)
    far, near = (A.kv_attention(q, f.cache, s, causal=causal, window=window) for s in f.seqs)
    seen = torch.arange(new, device=DEV) >= new - (64 - 1) if causal else torch.ones(new, dtype=torch.bool, device=DEV)
    assert torch.equal((near.abs().amax((1, 2)) > 0), seen) and torch.equal(far, near)


@pytest.mark.parametrize("P,D,n", [(16, 64, 1), (64, 128, 3), (256, 256, 20)])   # a wave a page; the workgroup
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mags", [
    [2.0e38, 3.38e38, 1.0e38, 3.38e38],           # the scale doubles, and 127 times it is above fp32's range
    [3.3895314e38, 3.3895314e38, 1.0, 0.0],       # bf16's largest
    [1.0e-38, 3.38e38, 3.38e38, 1e-30],
    [1.8e38, 3.0e38, 3.38e38],
])
def test_append_next_to_the_largest_numbers(A, P, D, n, dtype, mags):
    """127 times a page's scale may be infinite: everything finite has room then, and the scale stays."""
    cache = A.KVCache.empty(1, 1, P, D, device=DEV)
    codes, scales = np.zeros((1, 1, P, D), np.int8), np.zeros((1, 1), np.float32)
    table = np.zeros((1, 1), np.int32)
    for t, m in enumerate(mags):
        x = dev((np.linspace(-1, 1, n * D).reshape(n, 1, D) * m).astype(np.float32), dtype)
        assert bool(torch.isfinite(x).all())
        cu, lens = np.array([0, n]), np.array([n * (t + 1)])
        A.kv_append(x, x, cache, A.Sequences(dev(table), dev(cu, torch.int32), dev(lens, torch.int32)))
        with np.errstate(over="ignore"):
            R.append(x.float().cpu().numpy(), codes, scales, table, cu, lens, 1)
        torch.cuda.synchronize()
        assert np.isfinite(scales).all()
        assert np.array_equal(cache.k_scale.cpu().numpy(), scales) and np.array_equal(cache.v_scale.cpu().numpy(), scales), t
        assert np.array_equal(cache.k.cpu().numpy(), codes) and np.array_equal(cache.v.cpu().numpy(), codes), t


@pytest.mark.parametrize("new,lens,D,page", [([1, 2], [40, 300], 128, 32), ([20], [100], 64, 16), ([90, 40], [290, 60], 64, 16),
                                             ([100, 3], [150, 70], 128, 64), ([130], [130], 256, 32)])
@pytest.mark.parametrize("exps", [[-130], [-149, -131], [-126, -127, -128, -140], [-130, -122], [-149, -60, 0]])
def test_attention_with_subnormal_value_scales(A, new, lens, D, page, exps):
    """Value scales below fp32's normal range: each page counts with its own.  Codes are 64 to 127, so an output is
    2^6 of the largest scale or more: a normal fp32 number wherever that scale is 2^-131 or above."""
    rng = np.random.default_rng(D + len(exps))
    b = Batch(A, rng, new, lens, page)
    codes, scales, cache = random_cache(A, rng, b.pages, 2, page, D)
    codes[1] = rng.integers(64, 128, codes[1].shape).astype(np.int8)
    scales[1][:] = np.ldexp(np.float32(1), np.array(exps)[np.arange(b.pages) % len(exps)])[:, None]
    cache.v.copy_(dev(codes[1]))
    cache.v_scale.copy_(dev(scales[1]))
    for dtype in (BF, F32):
        q = dev((0.05 * rng.standard_normal((b.M, 4, D))).astype(np.float32), dtype)   # flat: every page weighs in
        check_tiny(A, q, b, codes, scales, cache)


def check_tiny(A, q, b, codes, scales, cache):
    """T.check_attention's bound, and half of the type's smallest step for outputs that are subnormal."""
    out = A.kv_attention(q, cache, b.seqs())
    ref, size, top, delta = R.attention(f64(q), codes[0], scales[0], codes[1], scales[1], b.table, b.cu, b.lens,
                                        q.shape[-1] ** -0.5, True, 0)
    wide = q.dtype == F32
    length = int(b.lens.max())
    e = ((q.shape[-1] + 16) * T.U + (2.0 ** -22 if wide else 0)) * delta
    bound = (2 * e + 8 * T.U + 2 * (length / 32 + 40) * T.U + 70 * T.U + (2.0 ** -21 if wide else 2.0 ** -11)) * size
    # a weight under fp16's range is off by half its step, 2^-25, of a largest one that stands at 2^8 at least
    bound = bound + 2.0 ** -33 * top + T.half_step(q.dtype) * (np.abs(ref) + bound) + torch.finfo(q.dtype).smallest_normal * T.half_step(q.dtype) * 2
    err = np.abs(f64(out) - ref)
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("new,dtype", [(1, BF), (1, F32), (90, BF), (90, F32)])
@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 13, 2.0 ** 16])
@pytest.mark.parametrize("page", [16, 64])
def test_pages_of_equal_large_scores_weigh_the_same(A, new, dtype, size, page):
    """Every key is the same, so all scores are, to the bit, whatever their size: a query's output is the mean of the
    values before it.  A probability is off by its fp16 half step (2^-11, for fp32 2^-22) and the rounding of an
    exponent of that size, 2^-24 size ln 2 (the fp32 kernels subtract equal numbers: none there)."""
    rng = np.random.default_rng(page)
    D, length = 128, 400
    b = Batch(A, rng, [new], [length], page)
    codes, scales, cache = random_cache(A, rng, b.pages, 1, page, D)
    codes[0][:] = rng.integers(-127, 128, D)
    scales[0][:] = 1.0 / 128
    cache.k.copy_(dev(codes[0]))
    cache.k_scale.copy_(dev(scales[0]))
    q = np.sign(codes[0][0, 0, 0].astype(np.float64)) * rng.uniform(0.5, 1, (new, 2, D))
    dot = (q * codes[0][0, 0, 0]).sum(-1).max() / 128
    q = dev(q.astype(np.float32), dtype)
    out = f64(A.kv_attention(q, cache, b.seqs(), scale=float(size / dot / np.log2(np.e))))
    t = np.arange(length)
    v = codes[1][b.table[0, t // page], 0, t % page] * scales[1][b.table[0, t // page], 0].astype(np.float64)[:, None]
    for i in range(new):
        seen = v[:length - new + i + 1]
        ref, mass = seen.mean(0), np.abs(seen).mean(0)
        weight = 2.0 ** -22 if dtype == F32 else 2.0 ** -11 + 2.0 ** -24 * size * np.log(2)
        # the sum of probabilities carries the exponent's part too; fp32 sums of 400 terms
        bound = (2 * weight + 2 * (length / 32 + 40) * T.U) * mass
        bound = bound + T.half_step(dtype) * (np.abs(ref) + bound)
        assert np.all(np.abs(out[i] - ref) <= bound), (i, float((np.abs(out[i] - ref) / bound).max()))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_angles_keep_their_low_bits(A, interleaved):
    """Heads of pairs (1, 0) become cosines and sines.  Near the half and the quarter turns, where one of the two is
    small, it has its own relative error: 2 ulp of the function, half of one for what the fp32 angle leaves out, 2^-53
    of the turn and of the angle on either side."""
    rng = np.random.default_rng(1)
    D = 256
    near = rng.choice([0.5, 0.25, -0.25, -0.5], D // 2) + rng.choice([-1, 1], D // 2) * np.exp(rng.uniform(np.log(1e-7), np.log(0.2), D // 2))
    freq = 2 * np.pi * near
    x = torch.zeros(3, 2, D, device=DEV)
    first = slice(0, D, 2) if interleaved else slice(0, D // 2)
    second = slice(1, D, 2) if interleaved else slice(D // 2, D)
    x[..., first] = 1
    pos = np.array([1, -1, 0], np.int32)
    y, _ = A.qk_norm_rope(x, None, dev(pos), dev(freq), interleaved=interleaved)
    angle = pos[:, None, None] * freq
    for got, ref in ((f64(y[..., first]), np.cos(angle)), (f64(y[..., second]), np.sin(angle))):
        err, bound = np.abs(got - ref), 2.5 * 2.0 ** -23 * np.abs(ref) + 4 * 2.0 ** -53 * np.pi
        assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("new,dtype", [([1, 1, 1], BF), ([5, 9, 6], F32), ([300, 20, 150], BF), ([100, 90, 3], F32)])
def test_workspace_behind_its_counters_may_hold_anything(A, new, dtype):
    rng = np.random.default_rng(6)
    b = Batch(A, rng, new, [3000, 700, 2000], 32)
    _, _, cache = random_cache(A, rng, b.pages, 2, 32, 128)
    q, seqs = dev(rng.standard_normal((b.M, 8, 128)).astype(np.float32), dtype), b.seqs()
    shape = (b.M, 3, 8, 2, 128)
    want = A.kv_attention(q, cache, seqs)
    filled = torch.full((A.kv_attention_workspace_bytes(*shape),), 255, dtype=torch.uint8, device=DEV)   # NaN as floats
    at = filled.data_ptr()
    filled[:A.COUNTER_BYTES] = 0
    assert torch.equal(A.kv_attention(q, cache, seqs, workspace=filled), want)
    # a new workspace costs its counters' zeros, not those of the megabytes behind them
    filled.fill_(255)
    del filled
    ws = A.kv_attention_workspace(*shape, DEV)
    if ws.data_ptr() != at:
        pytest.skip("the allocator gave other memory")
    assert int(ws[:A.COUNTER_BYTES].max()) == 0 and int(ws[A.COUNTER_BYTES:].min()) == 255
    assert torch.equal(A.kv_attention(q, cache, seqs, workspace=ws), want)


@pytest.mark.parametrize("count,D", [(1, 64), (1, 256), (300, 64), (300, 128)])    # units cut over workgroups; whole ones for waves
@pytest.mark.parametrize("dtype", [BF, F32])
def test_small_probabilities_of_single_tokens(A, count, D, dtype):
    """Two positions of a page, the second's probability 2^-18 to 2^-26 of the first's, whose value is 0: the output is the
    second's value at that weight.  The first's weight stands at 2^12 or more, so the second's has an fp16 half step, 2^-11 of
    itself or 2^-25: for fp32 queries two fp16 numbers, of which the second has the 2^-25."""
    rng = np.random.default_rng(D)
    b = Batch(A, rng, [1] * count, [2] * count, 16)
    codes = [np.zeros((b.pages, 8, 16, D), np.int8) for _ in range(2)]
    codes[0][:, :, 0, :64], codes[0][:, :, 1, :64] = 64, -64
    codes[1][:, :, 1] = rng.integers(64, 128, (b.pages, 8, D))
    scales = [np.full((b.pages, 8), 2.0 ** -6, np.float32), np.exp(rng.uniform(-2, 2, (b.pages, 8))).astype(np.float32)]
    cache = A.KVCache(dev(codes[0]), dev(codes[1]), dev(scales[0]), dev(scales[1]))
    gap = rng.uniform(18, 26, (count, 16)).astype(np.float32)       # in powers of two: 128 q sm_scale log2 e
    q = dev(np.repeat(gap[:, :, None] / 128, D, 2), dtype)
    sm = float(np.log(2))
    out = f64(A.kv_attention(q, cache, b.seqs(), scale=sm))
    gap = f64(q)[:, :, 0] * 128
    head = np.repeat(np.arange(8), 2)
    page = b.table[:, 0]
    p = 1 / (1 + 2.0 ** gap)
    value = codes[1][page][:, head, 1].astype(np.float64)
    sv = scales[1][page][:, head].astype(np.float64)[:, :, None]
    ref = p[:, :, None] * value * sv
    relative = (2.0 ** -22 if dtype == F32 else 2.0 ** -11) + (D + 16) * T.U * 27 + 80 * T.U
    bound = relative * ref + 2.0 ** -37 * value * sv
    bound = bound + T.half_step(dtype) * (ref + bound)
    err = np.abs(out - ref)
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("new,dtype", [([1, 1, 1], BF), ([6, 9, 2], BF), ([200, 30, 90], F32)])
def test_captured_without_a_workspace_of_its_own(A, new, dtype):
    """The graph zeroes its counters at every replay and follows lengths that change between them."""
    rng = np.random.default_rng(8)
    b = Batch(A, rng, new, [1500, 700, 900], 32, extra_width=0)
    _, _, cache = random_cache(A, rng, b.pages, 2, 32, 64)
    q, seqs = dev(rng.standard_normal((b.M, 8, 64)).astype(np.float32), dtype), b.seqs()
    A.kv_attention(q, cache, seqs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = A.kv_attention(q, cache, seqs)
    for turn in range(5):
        seqs.seq_lens.copy_(dev(rng.integers(1, 690, 3).astype(np.int32)))
        q.copy_(dev(rng.standard_normal(q.shape).astype(np.float32), dtype))
        graph.replay()
        want = A.kv_attention(q, cache, seqs)
        if turn % 2:
            torch.cuda.synchronize()
        assert torch.equal(out, want), turn


@pytest.mark.parametrize("new,lens,rows_behind", [
    ([1] * 30 + [500], list(range(100, 700, 20)) + [500], 0),          # single tokens in the prompt kernel
    ([1] * 70 + [300] + [1] * 5, list(range(20, 370, 5)) + [420] + [200] * 5, 7),    # a prompt in blocks of 32 rows
    ([1] * 90 + [120], [150] * 90 + [120], 0),                         # a prompt in blocks of 16 rows
    ([40, 0, 0, 0, 3] + [0] * 60, [200, 30, 0, 1, 90] + [0] * 60, 0),  # sequences without a token lower the average
    ([1, 1, 2], [300, 200, 100], 200),                                 # rows behind them raise it
])
@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64), (BF, 256)])
def test_batches_of_unlike_sequences(A, new, lens, rows_behind, dtype, D):
    rng = np.random.default_rng(len(new) + D)
    b = Batch(A, rng, new, lens, 32, rows_behind=rows_behind)
    codes, scales, cache = random_cache(A, rng, b.pages, 2, 32, D)
    q = dev((0.3 * rng.standard_normal((b.M, 8, D))).astype(np.float32), dtype)
    T.check_attention(A, q, b, codes, scales, cache)
