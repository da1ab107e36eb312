"""The serving operators on the GPU against their plain forms (tests/serving_ref.py).

Error bounds, u = 2^-24 (fp32), stated before the first run:

norm, int8   bit-exact: the factor is fp32 of a 64-bit mean, and fp64 sums in another order move it by one step
             in some 2^28 rows.
pages        whole numbers.
append       bit-exact.
attention    as tests/test_gpu_attention.py has it for the int8 cache, whose products and split these are: cached
             values are exact in both products.  delta bounds the score's sum of |terms|; its fp32 sum of D
             products is off by at most (D + 4) u delta, scaling and the exponent's argument by 4 u of the score
             and of the maximum each: e = (D + 16) u delta; fp32 queries as two fp16 numbers 2^-22 delta.  A
             weight is off by e + 4 u relatively, their sum too: 2 e + 8 u of A = sum p |v|.  Sums over
             positions: (L / 32 + 40) u A for numerator and denominator; joining at most 64 parts 70 u A.
             Probabilities as fp16: 2^-11 A (fp32: two numbers, 2^-21 A); what is under fp16's range is off by
             at most 2^-25, where the row's largest stands at 2^13 or more: 2^-38 of the largest weight (T).  The
             output's half step: 2^-8 (bf16) or 2^-24 of the value.
"""
import numpy as np
import pytest
import torch

import attention_ref
import oracle as O
import serving_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from w4a8_codebook_gemm_amd import serving
    serving.lib()
    return serving


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def f32(t):
    return t.detach().to(torch.float32).cpu().numpy()


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(DEV)


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ----------------------------------------------------------------------------- residual, norm, int8

def check_norm(S, x, r, w, eps, offset, got, normed):
    h = x.float() if r is None else (x.float() + r.float()).to(r.dtype)
    if r is not None:
        assert got.h.dtype == r.dtype and torch.equal(got.h, h)
    y = R.norm(f32(h), f32(w), eps, offset)
    if normed is not None:
        assert got.normed.dtype == normed and torch.equal(got.normed.cpu(), torch.from_numpy(y).to(normed))
    if got.x_q is not None:
        xq, sx = O.prepare(y)
        assert np.array_equal(got.s_x.cpu().numpy(), sx) and np.array_equal(got.x_q.cpu().numpy(), xq)


NORM = [
    # M, K, x, residual, normed, padded rows
    (1, 256, F32, None, None, 0),
    (1, 5120, F32, BF, None, 0),
    (1, 5120, BF, F32, F32, 0),
    (3, 512, BF, BF, BF, 8),
    (7, 768, F32, F32, None, 264),
    (61, 5120, BF, BF, BF, 0),
    (300, 1280, F32, BF, F32, 0),
    (2, 16384, F32, F32, None, 0),          # a lane has one block
    (3, 16640, BF, F32, BF, 16),            # two blocks
    (2, 17408, F32, None, None, 0),
    (2, 32768, BF, BF, None, 0),
    (3, 33024, F32, BF, F32, 8),            # up to four
    (2, 65536, F32, F32, BF, 0),
    (4099, 256, BF, F32, None, 0),          # more tokens than workgroups
    (2500, 2048, F32, BF, BF, 0),
    (4097, 5120, F32, BF, BF, 0),           # three blocks a lane group, two tokens a workgroup
    (4096, 2816, BF, F32, None, 24),        # one wave a token, with a block to spare
    (4100, 9216, BF, BF, None, 0),          # three waves a token
    (4099, 1536, F32, F32, None, 0),
]


@pytest.mark.parametrize("M,K,xdt,rdt,normed,pad", NORM)
def test_add_norm_prepare(S, M, K, xdt, rdt, normed, pad):
    g = torch.Generator(device=DEV).manual_seed(M + K)
    x = torch.randn(M, K + pad, generator=g, device=DEV).to(xdt)[:, :K]
    r = None if rdt is None else (torch.randn(M, K + pad, generator=g, device=DEV) * 20).to(rdt)[:, :K]
    w = torch.randn(K, generator=g, device=DEV) * 0.3
    got = S.add_norm_prepare(x, w, r, eps=1e-6, weight_offset=1.0, normed_dtype=normed)
    check_norm(S, x, r, w, 1e-6, 1.0, got, normed)


def test_add_norm_in_place_and_norm_alone(S):
    """The residual updated in place, x as the output where types agree, and the norm without its int8 form."""
    M, K = 37, 1024
    x, r, w = torch.randn(M, K, device=DEV), torch.randn(M, K, device=DEV), torch.rand(K, device=DEV)
    want = S.add_norm_prepare(x, w, r, normed_dtype=BF)
    for target in ("r", "x"):
        a, b = x.clone(), r.clone()
        got = S.add_norm_prepare(a, w, b, h_out=b if target == "r" else a)
        assert torch.equal(got.h, want.h) and torch.equal(got.x_q, want.x_q) and torch.equal(got.s_x, want.s_x)
        assert torch.equal(a if target == "r" else b, x if target == "r" else r)
    alone = S.add_norm_prepare(x, w, r, normed_dtype=BF, quantise=False)
    assert alone.x_q is None and torch.equal(alone.normed, want.normed) and torch.equal(alone.h, want.h)
    first = S.add_norm_prepare(x, w)
    assert first.h is None and first.normed is None
    check_norm(S, x, None, w, 1e-6, 0.0, first, None)


def test_add_norm_of_rows_that_are_zero_or_not_finite(S):
    M, K = 9, 512
    x, r, w = torch.randn(M, K, device=DEV), torch.randn(M, K, device=DEV), torch.rand(K, device=DEV)
    want = S.add_norm_prepare(x, w, r, normed_dtype=F32)
    x[2] = 0
    r[2] = 0
    r[4, 7] = float("nan")
    x[6, 500] = float("inf")
    got = S.add_norm_prepare(x, w, r, normed_dtype=F32)
    rest = [0, 1, 3, 5, 7, 8]
    for a, b in zip(got, want):
        assert torch.equal(a[rest], b[rest])
    assert float(got.s_x[2]) == 0 and int(got.x_q[2].abs().max()) == 0 and float(got.normed[2].abs().max()) == 0


@pytest.mark.parametrize("mag", [1e-30, 1e-15, 1e15])
def test_add_norm_magnitudes(S, mag):
    """Squares far outside fp32's range: the sum is a 64-bit one."""
    x, r = (torch.randn(5, 768, device=DEV) * mag for _ in range(2))
    w = torch.randn(768, device=DEV)
    got = S.add_norm_prepare(x, w, r, eps=0.0, normed_dtype=F32)
    check_norm(S, x, r, w, 0.0, 0.0, got, F32)


# ----------------------------------------------------------------------------- pages

def make_pages(S, rng, lens, width, page, spare):
    """Sequences that hold pages in random order, the others free."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), width), -7, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    free = np.full(pages, 12345, np.int32)
    free[:spare] = order[at:]
    return dict(table=table, lens=np.array(lens, np.int32), free=free, count=spare)


def on_gpu(S, p, page):
    return S.Pages(dev(p["table"]), dev(p["lens"]), dev(p["free"]), i32(p["count"]), page)


def check_assign(S, p, new, page, M, in_place):
    pages = on_gpu(S, p, page)
    b, width = p["table"].shape
    new = np.array(new, np.int32)
    out = None if in_place else S.Batch.empty(b, M, DEV)
    got = S.pages_assign(pages, dev(new), M, out=out)
    torch.cuda.synchronize()
    table, cu, lens, positions, slots, count, missing = R.assign(p["table"], p["lens"], p["free"], p["count"], new, page, M)
    assert np.array_equal(pages.page_table.cpu().numpy(), table)
    assert np.array_equal(pages.free_pages.cpu().numpy(), p["free"])
    for a, want in ((got.cu_tokens, cu), (got.seq_lens, lens), (got.positions, positions), (got.slots, slots),
                    (got.free_count, [count]), (got.missing, [missing])):
        assert np.array_equal(a.cpu().numpy(), want)
    if in_place:
        assert got.seq_lens is pages.seq_lens and got.free_count is pages.free_count
    else:
        assert np.array_equal(pages.seq_lens.cpu().numpy(), p["lens"]) and int(pages.free_count) == p["count"]
    return pages, got


ASSIGN = [
    # lens, new, page, width, spare, rows behind the last token
    ([0], [1], 16, 4, 3, 0),
    ([0], [0], 16, 1, 1, 1),
    ([15, 16, 17, 0, 31], [1, 1, 1, 1, 2], 16, 8, 9, 2),
    ([5, 0, 100, 33], [0, 300, 0, 40], 32, 16, 30, 0),
    ([5, 0, 100, 33], [300, 300, 7, 40], 64, 20, 8, 5),          # the list runs out
    ([5, 0, 100, 33], [30, 30, 70, 40], 16, 20, 0, 0),           # it is empty
    ([60, 10, 64, 3], [10, 100, 1, 1], 16, 4, 40, 0),            # tokens behind the tables
    ([0, 3, 0], [2500, 0, 3000], 16, 200, 400, 7),               # more tokens than one workgroup takes
    ([0] * 70, [200] * 70, 256, 3, 80, 100),
]


@pytest.mark.parametrize("lens,new,page,width,spare,behind", ASSIGN)
@pytest.mark.parametrize("in_place", [False, True])
def test_assign(S, lens, new, page, width, spare, behind, in_place):
    p = make_pages(S, np.random.default_rng(sum(new) + page), lens, width, page, spare)
    check_assign(S, p, new, page, sum(new) + behind, in_place)


@pytest.mark.parametrize("count,hi,ctx,page", [(61, 1, 4000, 64), (1023, 3, 60, 16), (1024, 1, 100, 16), (1025, 9, 100, 16),
                                               (2500, 40, 200, 16), (5000, 1, 30, 32)])
@pytest.mark.parametrize("in_place", [False, True])
def test_assign_many(S, count, hi, ctx, page, in_place):
    rng = np.random.default_rng(count)
    lens, new = rng.integers(0, ctx + 1, count), rng.integers(0, hi + 1, count)
    p = make_pages(S, rng, list(lens), -(-(ctx + hi) // page), page, int(new.sum()) // page + count // 2)
    check_assign(S, p, new, page, int(new.sum()) + 3, in_place)


def test_assign_numbers_out_of_range(S):
    """Lengths, counts, new tokens and pages that a broken program could leave; fewer rows than tokens."""
    rng = np.random.default_rng(1)
    p = make_pages(S, rng, [20, 40, 7], 5, 16, 9)
    p["lens"] = np.array([-5, 2 ** 31 - 1, 7], np.int32)
    p["table"][2, 0] = 2 ** 31 - 1
    for count in (-3, 2 ** 31 - 1, 4):
        p["count"] = count
        check_assign(S, p, [30, 3, 20], 16, 64, False)
        check_assign(S, p, [-(2 ** 31), 2 ** 31 - 1, 5], 16, 64, True)
    p["count"] = 9
    for rows in (1, 3, 20, 30, 31, 45):
        check_assign(S, p, [30, 1, 20], 16, rows, False)
    p["free"][:9] = [-1, 2 ** 31 - 1, -(2 ** 31), 3, 4, 5, -7, 10 ** 6, 1]     # numbers of no page
    check_assign(S, p, [100, 1, 20], 16, 140, True)


@pytest.mark.parametrize("M", [50, 700, 5000])
@pytest.mark.parametrize("in_place", [False, True])
def test_assign_more_tokens_than_rows(S, M, in_place):
    """Sums of new tokens that pass 32 bits, the rows used up by any of the sequences."""
    rng = np.random.default_rng(M)
    count = 2500
    p = make_pages(S, rng, list(rng.integers(0, 40, count)), 4, 16, 2000)
    most = np.full(count, 2 ** 31 - 1, np.int32)
    few = rng.integers(0, 2, count).astype(np.int32)
    for new in (most, few, np.where(np.arange(count) < 1400, few, most)):
        check_assign(S, p, new, 16, M, in_place)


def test_assign_as_many_rows_as_there_may_be(S):
    M, B, width = 2 ** 24, 1100, 2 ** 21 // 256
    pages = S.Pages.empty(B, width, 9000, 256, DEV)
    new = torch.full((B,), 2 ** 31 - 1, dtype=torch.int32, device=DEV)
    new[:3] = i32(5, 0, 2 ** 21)
    out = S.pages_assign(pages, new, M, out=S.Batch.empty(B, M, DEV))
    torch.cuda.synchronize()
    assert out.cu_tokens.tolist() == [0, 5, 5, 5 + 2 ** 21] + [M] * (B - 3)
    assert out.seq_lens.tolist() == [5, 0, 2 ** 21, 2 ** 21] + [0] * (B - 4)   # the fourth's table ends at 2^21
    rest = M - 5 - 2 ** 21
    # 1 + 8192 pages, then 807 of the fourth's 8192, whose tokens want rest / 256 pages
    assert int(out.free_count) == 0 and int(out.missing) == 8193 + -(-rest // 256) - 9000
    assert torch.equal(out.positions[5 + 2 ** 21:], torch.arange(rest, dtype=torch.int32, device=DEV))
    held = torch.cat([torch.arange(5, device=DEV), 256 + torch.arange(2 ** 21 + 807 * 256, device=DEV)])
    assert torch.equal(out.slots[:held.numel()], held) and bool((out.slots[held.numel():] == -1).all())


RELEASE = [
    ([1], [0], 16), ([0], [5], 16), ([100, 17, 64], [33, 16, 64], 16), ([100, 17, 64], [-4, 500, 1], 32),
    ([3000, 2999, 1], [0, 0, 0], 16),
]


def check_release(S, p, keep, page, in_place):
    pages = on_gpu(S, p, page)
    keep = np.array(keep, np.int32)
    lens, count = S.pages_release(pages, dev(keep), in_place=in_place)
    torch.cuda.synchronize()
    free, want, n = R.release(p["table"], p["lens"], p["free"], p["count"], keep, page)
    assert np.array_equal(pages.free_pages.cpu().numpy(), free)
    assert np.array_equal(lens.cpu().numpy(), want) and int(count) == n
    assert np.array_equal(pages.page_table.cpu().numpy(), p["table"])
    if in_place:
        assert lens is pages.seq_lens and count is pages.free_count
    else:
        assert np.array_equal(pages.seq_lens.cpu().numpy(), p["lens"]) and int(pages.free_count) == p["count"]
    return pages


@pytest.mark.parametrize("lens,keep,page", RELEASE)
@pytest.mark.parametrize("in_place", [False, True])
def test_release(S, lens, keep, page, in_place):
    p = make_pages(S, np.random.default_rng(sum(lens)), lens, max(-(-n // page) for n in lens) + 1, page, 5)
    check_release(S, p, keep, page, in_place)
    p["table"][0, ::3] = -1                      # pages given up
    p["table"][-1, 0] = len(p["free"])
    check_release(S, p, keep, page, in_place)


@pytest.mark.parametrize("count,ctx,page", [(61, 4000, 64), (1024, 100, 16), (1500, 700, 16), (4000, 40, 16)])
def test_release_many(S, count, ctx, page):
    rng = np.random.default_rng(count)
    lens = rng.integers(0, ctx + 1, count)
    keep = np.where(rng.random(count) < 0.3, 0, lens - rng.integers(0, 60, count))
    p = make_pages(S, rng, list(lens), -(-ctx // page) + 1, page, 11)
    check_release(S, p, keep, page, True)
    p["table"][rng.random(p["table"].shape) < 0.2] = -1
    check_release(S, p, keep, page, False)


@pytest.mark.parametrize("count", [1023, 1024, 2050])
@pytest.mark.parametrize("every", [1, 2, 65])
def test_release_of_a_page_each(S, count, every):
    """Each sequence, or one in `every`, gives back one page; the last of them many."""
    rng = np.random.default_rng(count + every)
    lens = rng.integers(17, 33, count)
    lens[count - 2] = 5000
    keep = np.where(np.arange(count) % every == 0, 16, lens)
    keep[count - 2] = 20
    p = make_pages(S, rng, [int(x) for x in lens], 320, 16, 3)
    check_release(S, p, keep, 16, False)


def test_release_into_a_list_without_room(S):
    """A program that gives a page back twice: the list's end is not passed."""
    p = make_pages(S, np.random.default_rng(2), [100, 90], 8, 16, 3)
    p["table"][1, :6] = p["table"][0, :6]
    p["count"] = 10
    check_release(S, p, [0, 0], 16, True)


def test_assign_and_release_undo_each_other(S):
    """A hundred steps of growth, refused drafts and ends: no page is lost, none is held twice."""
    rng = np.random.default_rng(3)
    B, page, total = 40, 16, 700
    pages = S.Pages.empty(B, 40, total, page, DEV)
    for step in range(100):
        lens = pages.seq_lens.cpu().numpy()
        new = np.minimum(rng.integers(0, 40 if step % 10 == 0 else 5, B), 600 - lens).astype(np.int32)
        before = [t.clone() for t in (pages.free_pages, pages.free_count)]
        b = S.pages_assign(pages, dev(new), 2000)
        if step % 7 == 0:                         # all of it refused: the list is what it was
            S.pages_release(pages, dev(lens))
            assert torch.equal(before[0], pages.free_pages) and torch.equal(before[1], pages.free_count)
            continue
        assert int(b.missing) == 0
        keep = np.where(rng.random(B) < 0.1, 0, lens + rng.integers(0, new + 1)).astype(np.int32)
        S.pages_release(pages, dev(keep))
        lens, table = pages.seq_lens.cpu().numpy(), pages.page_table.cpu().numpy()
        assert np.array_equal(lens, keep)
        held = np.concatenate([table[i, :-(-n // page)] for i, n in enumerate(lens)])
        free = pages.free_pages.cpu().numpy()[:int(pages.free_count)]
        assert np.array_equal(np.sort(np.concatenate([held, free])), np.arange(total))


def test_pages_captured_and_replayed(S):
    """Growth in place, in a graph: every replay goes on from where the last one ended."""
    for B, M in ((5, 5), (90, 6000)):             # one launch; two
        new = torch.full((B,), M // B, dtype=torch.int32, device=DEV)
        eager, cap = (S.Pages.empty(B, 60, 60 * B, 16, DEV) for _ in range(2))
        S.pages_assign(S.Pages.empty(B, 60, 60 * B, 16, DEV), new, M)
        out = S.Batch.empty(B, M, DEV, cap.seq_lens, cap.free_count)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            S.pages_assign(cap, new, M, out=out)
        for turn in range(6):
            want = S.pages_assign(eager, new, M)
            graph.replay()
            if turn % 2:
                torch.cuda.synchronize()
            for name in ("cu_tokens", "seq_lens", "positions", "slots", "free_count", "missing"):
                assert torch.equal(getattr(out, name), getattr(want, name)), (turn, name)
            assert torch.equal(cap.page_table, eager.page_table)


# ----------------------------------------------------------------------------- the append

def random_cache(S, rng, pages, hkv, page, d, units=None):
    """Codes and scale bytes of every kind, and units of several sizes."""
    n = lambda *shape: rng.integers(0, 256, shape).astype(np.uint8)  # noqa: E731
    k, v = n(pages, hkv, page, d // 2), n(pages, hkv, page, d // 2)
    ks, vs = n(pages, hkv, page, d // 16), n(pages, hkv, d // 16, page)
    if units is None:
        units = [2.0 ** rng.integers(-20, -17, hkv) * rng.uniform(1, 2, hkv) for _ in range(2)]
    units = [np.asarray(u, np.float32) for u in units]
    # scales within a factor of 16 of each other, so that no position alone decides
    ks, vs = 128 + ks % 64, 128 + vs % 64
    return S.KV4Cache(*(dev(x) for x in (k, v, ks, vs, *units)))


def host(c):
    return {n: getattr(c, n).cpu().numpy() for n in ("k", "v", "k_scale", "v_scale", "k_unit", "v_unit")}


def dense(c):
    """The cache's keys and values in 64 bits, [pages, heads, page, D]."""
    h = host(c)
    return R.values4(h["k"], h["k_scale"], h["k_unit"]), R.values4(h["v"], h["v_scale"].transpose(0, 1, 3, 2), h["v_unit"])


def check_append(S, cache, k, v, slots):
    want = host(cache)
    S.kv4_append(k, v, cache, dev(slots))
    torch.cuda.synchronize()
    P = cache.k.shape[2]
    kc, ks = R.quantise4(f32(k), want["k_unit"])
    vc, vs = R.quantise4(f32(v), want["v_unit"])
    for i, s in enumerate(slots):
        if 0 <= s < cache.k.shape[0] * P:
            p, at = divmod(int(s), P)
            want["k"][p, :, at], want["k_scale"][p, :, at] = kc[i], ks[i]
            want["v"][p, :, at], want["v_scale"][p, :, :, at] = vc[i], vs[i]
    got = host(cache)
    for name in want:
        assert np.array_equal(got[name], want[name]), name


APPEND = [
    # M, Hkv, D, page, dtype, magnitude
    (1, 1, 64, 16, BF, 1.0),
    (1, 4, 256, 64, F32, 1.0),
    (15, 2, 128, 16, F32, 30.0),
    (16, 3, 64, 32, BF, 1e-3),
    (17, 5, 256, 128, BF, 100.0),
    (61, 4, 256, 64, BF, 1.0),
    (333, 8, 128, 256, F32, 1e4),
    (1000, 1, 64, 16, F32, 1e-6),
]


@pytest.mark.parametrize("M,Hkv,D,page,dtype,mag", APPEND)
def test_append(S, M, Hkv, D, page, dtype, mag):
    rng = np.random.default_rng(M + D)
    pages = M // page + 3
    cache = random_cache(S, rng, pages, Hkv, page, D, [rng.uniform(0.5, 4, Hkv) * 2.0 ** -14 for _ in range(2)])
    x = [dev((rng.standard_normal((M, 2 * Hkv, D)) * mag * np.exp(rng.uniform(-4, 0, (M, 2 * Hkv, 1)))).astype(np.float32),
             dtype)[:, i * Hkv:(i + 1) * Hkv] for i in (0, 1)]
    x[0][0, 0] = 0
    x[1][0, 0, ::2] = -0.0
    slots = rng.permutation(pages * page)[:M]
    slots[M // 2] = -1
    if M > 3:
        slots[1], slots[2] = pages * page, 2 ** 62
    check_append(S, cache, x[0], x[1], slots)


def test_append_rounds_at_every_border(S):
    """Values on and next to the borders between codes and between scales."""
    D, H, unit = 64, 2, 2.0 ** -14
    cache = S.KV4Cache.empty(40, H, 16, D, DEV)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    near = np.concatenate([np.nextafter(mids.astype(np.float32), np.float32(0)), mids, np.nextafter(mids.astype(np.float32), np.float32(9))])
    rows = []
    for byte in list(range(1, 40)) + [63, 64, 100, 200, 254, 255]:
        step = R.STEPS[byte] * unit
        x = np.zeros(D)
        x[::16] = 6 * step                                    # each group's largest: this byte
        x[1:16], x[17:32], x[33:48] = np.resize(near, 15) * step, -np.resize(near[::-1], 15) * step, near[6:21] * step
        rows.append(x)
    for byte in (1, 2, 14, 15, 16, 17, 31, 32, 33, 47, 48, 253, 254):      # halfway between two scales, and next to it
        mid = np.float32(6 * (R.STEPS[byte] + R.STEPS[byte + 1]) / 2 * unit)
        for m in (np.nextafter(mid, np.float32(0)), mid, np.nextafter(mid, np.float32(1e9))):
            rows.append(np.linspace(-1, 1, D) * np.float64(m))
    rows += [np.full(D, v) for v in (0.0, -0.0, 1e-45, -1e-45, 1e-30, unit * 0.24, unit * 3, unit * 2.9999, 3.4e38, -3.4e38, 1e20)]
    x = np.stack(rows).astype(np.float32)
    x = np.stack([x, -x], 1)
    check_append(S, cache, dev(x), dev(x[:, ::-1].copy()), np.arange(len(x)) + 5)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_of_values_that_are_not_finite(S, dtype):
    """An infinity counts as the largest magnitude; a NaN spoils its own value and nothing else."""
    rng = np.random.default_rng(7)
    x = rng.standard_normal((20, 2, 128)).astype(np.float32)
    a, b = (S.KV4Cache.empty(2, 2, 16, 128, DEV) for _ in range(2))
    S.kv4_append(dev(x, dtype), dev(x, dtype), a, torch.arange(20, device=DEV))
    y = x.copy()
    y[3, 1, 20] = np.nan
    x2 = x.copy()
    x2[3, 1, 20] = 0.0
    S.kv4_append(dev(y, dtype), dev(x2, dtype), b, torch.arange(20, device=DEV))
    h = host(b)
    same = h["k"][0, 1, 3] == h["v"][0, 1, 3]
    assert same.sum() == 63 and not same[10] and (h["k"][0, 1, 3, 10] ^ h["v"][0, 1, 3, 10]) >> 4 == 0
    assert np.array_equal(h["k_scale"], h["v_scale"].transpose(0, 1, 3, 2))
    y[3, 1, 20] = -np.inf
    check_append(S, b, dev(y, dtype), dev(y, dtype), np.arange(20))


# ----------------------------------------------------------------------------- attention

class Batch:
    """Sequences with pages in random order; new tokens and lengths as given."""

    def __init__(self, rng, new, lens, page, extra_width=1, spare=2, rows_behind=0):
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

    def seqs(self):
        from w4a8_codebook_gemm_amd.attention import Sequences
        return Sequences(dev(self.table), dev(self.cu), dev(self.lens))


def check_attention(S, q, b, cache, causal=True, window=0, workspace=None, scale=None, out=None):
    d = q.shape[-1]
    sm = d ** -0.5 if scale is None else scale
    if out is None:
        out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
        S.kv4_attention(q, cache, b.seqs(), scale=sm, causal=causal, window=window, workspace=workspace, out=out)
        torch.cuda.synchronize()
    k, v = dense(cache)
    one = np.ones(k.shape[:2])
    ref, size, top, delta = attention_ref.attention(f64(q), k, one, v, one, b.table, b.cu, b.lens, sm, causal, window)
    for i in range(len(b.lens)):                          # tokens in front of position 0 see nothing
        n = int(b.cu[i + 1] - b.cu[i])
        front = slice(int(b.cu[i]), int(b.cu[i]) + max(0, n - max(int(b.lens[i]), 0)))
        for x in (ref, size, top, delta):
            x[front] = 0
    got = f64(out)
    behind = np.isnan(ref)
    assert np.all(got[behind] == 7.0)                     # rows of no sequence
    ref = np.where(behind, 7.0, ref)
    wide = q.dtype == F32
    length = int(max(b.lens.max(), 1))
    e = ((d + 16) * U + (2.0 ** -22 if wide else 0)) * delta
    bound = (2 * e + 8 * U + 2 * (length / 32 + 40) * U + 70 * U + (2.0 ** -21 if wide else 2.0 ** -11)) * size
    # a row's largest probability so far stands at 2^10 or more (2^14, less 1 for a whole maximum and 3 by which that grows ahead);
    # where fp16 numbers have no more bits, from 2^-14 down, they are 2^-24 apart: half of it is 2^-35 of the largest
    bound = bound + 2.0 ** -35 * top + half_step(q.dtype) * (np.abs(ref) + bound)
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
    ([9, 3], [60, 300], 8, 2, 64, 128, BF, True, 0),
    ([130, 65, 1], [130, 200, 50], 6, 2, 128, 32, BF, True, 0),
    ([200], [517], 12, 2, 256, 64, BF, True, 0),
    ([100, 3], [150, 300], 4, 2, 256, 16, F32, True, 0),
    ([257, 64], [257, 64], 4, 4, 64, 64, BF, True, 50),
    ([150], [400], 8, 2, 128, 128, F32, True, 1),
    ([90, 120], [90, 333], 3, 1, 128, 32, F32, False, 0),
    ([10, 300], [4, 290], 2, 1, 64, 16, BF, True, 0),       # first rows stand in front of position 0
    ([10, 300], [4, 290], 2, 1, 64, 16, F32, False, 0),
    ([7, 1], [3, 9], 2, 2, 256, 16, BF, False, 0),
    ([70], [700], 5, 1, 256, 256, BF, True, 200),
    ([80, 90], [300, 95], 4, 1, 64, 16, F32, True, 0),
]


@pytest.mark.parametrize("new,lens,Hq,Hkv,D,page,dtype,causal,window", ATTN)
def test_attention(S, new, lens, Hq, Hkv, D, page, dtype, causal, window):
    rng = np.random.default_rng(sum(lens) + D)
    b = Batch(rng, new, lens, page, rows_behind=2)
    cache = random_cache(S, rng, b.pages, Hkv, page, D)
    q = dev(rng.standard_normal((b.M, 2 * Hq, D)).astype(np.float32) * 2, dtype)[:, Hq:]
    check_attention(S, q, b, cache, causal, window)


@pytest.mark.parametrize("new,lo,hi,count,Hq,Hkv,D,dtype", [
    (1, 500, 6000, 40, 24, 4, 256, BF),       # several units and parts of units for a workgroup, blocks of 16 rows
    (1, 20, 1500, 300, 8, 8, 64, F32),        # more sequences than a wave has lanes
    (7, 300, 2500, 40, 12, 3, 128, BF),       # blocks of 32 rows
    (60, 60, 1200, 70, 8, 2, 128, BF),        # many rows, more sequences than lanes
    (90, 90, 900, 10, 8, 2, 256, F32),
])
def test_attention_of_many_units(S, new, lo, hi, count, Hq, Hkv, D, dtype):
    """Batches large enough that a workgroup has several units, cut anywhere."""
    rng = np.random.default_rng(D + count)
    lens = rng.integers(lo, hi, count)
    b = Batch(rng, [new] * count, list(lens), 16)
    cache = random_cache(S, rng, b.pages, Hkv, 16, D)
    q = dev(rng.standard_normal((b.M, Hq, D)).astype(np.float32), dtype)
    check_attention(S, q, b, cache)


@pytest.mark.parametrize("new,Hq,Hkv", [(3, 64, 8), (6, 64, 8), (2, 32, 32), (9, 12, 4)])
@pytest.mark.parametrize("D,page,window", [(64, 16, 0), (64, 64, 70), (128, 16, 90), (128, 32, 0), (256, 16, 0), (256, 32, 33)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_of_drafts(S, new, Hq, Hkv, D, page, window, dtype):
    """Sequences of unlike lengths with 2 to 48 rows, in blocks of 16 and of 32; pages given up, lengths shorter than the draft."""
    rng = np.random.default_rng(new + D)
    count = 17
    lens = [int(x) for x in rng.integers(new, 400, count)]
    lens[3], lens[9], lens[10] = new - 1, new, 1100
    news = [new] * count
    news[5] = 0
    b = Batch(rng, news, lens, page, rows_behind=new)
    cache = random_cache(S, rng, b.pages, Hkv, page, D)
    b.table[7, 0] = -1
    b.table[11] = b.pages
    q = dev(rng.standard_normal((b.M, Hq, D)).astype(np.float32), dtype)
    check_attention(S, q, b, cache, window=window)


@pytest.mark.parametrize("count,lo,hi,Hq,Hkv,D,page,dtype,window", [
    (300, 1, 60, 16, 8, 64, 16, BF, 0),
    (300, 30, 260, 24, 8, 128, 32, F32, 0),
    (150, 40, 90, 32, 16, 256, 16, BF, 33),
])
@pytest.mark.parametrize("shape", ["alike", "some empty", "one long", "several tokens"])
def test_attention_of_many_short_sequences(S, count, lo, hi, Hq, Hkv, D, page, dtype, window, shape):
    rng = np.random.default_rng(count + D)
    new, lens = [1] * count, [int(x) for x in rng.integers(lo, hi, count)]
    if shape == "some empty":
        new = [int(x) for x in rng.integers(0, 2, count)]
    elif shape == "one long":
        lens[count // 3] = 9000
    elif shape == "several tokens":
        new = [min(int(x), 16 * Hkv // Hq) for x in rng.integers(1, 4, count)]
    b = Batch(rng, new, lens, page, rows_behind=3)
    cache = random_cache(S, rng, b.pages, Hkv, page, D)
    b.table[5, 0] = -1
    b.table[7] = -1
    q = dev(rng.standard_normal((b.M, Hq, D)).astype(np.float32), dtype)
    check_attention(S, q, b, cache, window=window)


@pytest.mark.parametrize("new,lens,Hq,Hkv,D,window", [
    ([600] * 5, [600] * 5, 16, 16, 64, 0),                 # a workgroup for each block of rows and head
    ([20] * 70, [90 + i for i in range(70)], 8, 2, 128, 0),  # the same of more sequences than a wave has lanes
    ([150, 0, 90, 0, 200, 64], [180, 9, 90, 0, 231, 300], 8, 4, 128, 100),
    ([0] * 64 + [90, 40], [5] * 64 + [120, 200], 4, 2, 256, 0),
    ([90] * 3 + [100], [90] * 3 + [3000], 8, 2, 64, 0),    # one is long: cut
])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_of_whole_blocks(S, new, lens, Hq, Hkv, D, window, dtype):
    rng = np.random.default_rng(sum(new))
    b = Batch(rng, new, lens, 32, rows_behind=3)
    cache = random_cache(S, rng, b.pages, Hkv, 32, D)
    q = dev(rng.standard_normal((b.M, Hq, D)).astype(np.float32), dtype)
    check_attention(S, q, b, cache, window=window)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("new", [[1, 1, 1], [40, 90, 20]])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_pages_given_up(S, dtype, new, D):
    """Pages marked -1, past the cache, or all of a sequence's."""
    rng = np.random.default_rng(3)
    b = Batch(rng, new, [200, 300, 90], 16)
    b.table[0, 2] = -1
    b.table[0, 5:8] = 2 ** 31 - 1
    b.table[1, 0] = b.pages
    b.table[2, :6] = -1
    cache = random_cache(S, rng, b.pages, 2, 16, D)
    q = dev(rng.standard_normal((b.M, 6, D)).astype(np.float32), dtype)
    check_attention(S, q, b, cache)
    check_attention(S, q, b, cache, window=40)


def test_offsets_and_lengths_out_of_range(S):
    """Offsets and lengths that a broken program could leave: held to their range."""
    from w4a8_codebook_gemm_amd.attention import Sequences
    rng = np.random.default_rng(4)
    cache = random_cache(S, rng, 8, 1, 16, 64)
    b = Batch(rng, [3, 3], [20, 30], 16, extra_width=0, spare=4)
    b.lens[1] = 10 ** 6                 # held to the table's width
    q = dev(rng.standard_normal((6, 2, 64)).astype(np.float32))
    check_attention(S, q, b, cache)
    bad = Sequences(dev(b.table), dev(np.array([-5, 4, 2 ** 31 - 1], np.int32)), dev(np.array([-3, 2 ** 31 - 1], np.int32)))
    out = S.kv4_attention(q, cache, bad)
    torch.cuda.synchronize()
    assert torch.equal(out[:4], torch.zeros_like(out[:4]))


@pytest.mark.parametrize("new,lens", [([1, 1], [300, 40]), ([60, 9], [200, 70]), ([3, 9], [200, 70])])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 256])
def test_attention_of_every_byte(S, new, lens, dtype, D):
    """Scale bytes from 0 to 255, units at both ends of their range, sharp and flat softmaxes."""
    rng = np.random.default_rng(9)
    for ku, vu, qs in ((2.0 ** -24, 2.0 ** -14, 4.0), (2.0 ** -120, 2.0 ** -120, 0.0), (2.0 ** -30, 2.0 ** 90, 1.0), (2.0 ** -20, 1.0, 1.0)):
        b = Batch(rng, new, lens, 16)
        cache = random_cache(S, rng, b.pages, 1, 16, D, [[ku], [vu]])
        cache.k_scale.copy_(dev(rng.integers(0, 256, cache.k_scale.shape).astype(np.uint8)))
        cache.v_scale.copy_(dev(rng.integers(0, 256, cache.v_scale.shape).astype(np.uint8)))
        q = dev(rng.standard_normal((b.M, 2, D)).astype(np.float32) * qs, dtype)
        check_attention(S, q, b, cache, scale=0.125)
        check_attention(S, q, b, cache, scale=-0.02)


@pytest.mark.parametrize("new,lens,D,page,window", [
    ([3, 1], [130, 40], 128, 16, 0),
    ([3, 1], [130, 140], 256, 32, 20),
    ([20, 1], [200, 60], 64, 16, 30),
    ([90, 40], [290, 60], 128, 16, 0),
    ([70, 80], [400, 80], 256, 16, 33),
    ([300, 2], [300, 9], 64, 64, 0),
])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_of_what_is_not_seen(S, new, lens, D, page, window, dtype):
    """Slots behind a sequence's end and other rows' queries may hold anything: a row's bits stay."""
    rng = np.random.default_rng(D + window)
    b = Batch(rng, new, lens, page)
    cache = random_cache(S, rng, b.pages, 2, page, D)
    q = dev(rng.standard_normal((b.M, 6, D)).astype(np.float32), dtype)
    seqs = b.seqs()
    want = S.kv4_attention(q, cache, seqs, window=window)
    assert bool(torch.isfinite(want).all())
    used = np.zeros((b.pages, page), bool)
    for s, n in enumerate(lens):
        used[b.table[s, np.arange(n) // page], np.arange(n) % page] = True
    un = dev(~used)[:, None, :].expand(-1, 2, -1)
    for byte in (0, 255):
        for t in (cache.k, cache.v, cache.k_scale):
            t[un] = byte
        cache.v_scale.transpose(2, 3)[un] = byte
        assert torch.equal(S.kv4_attention(q, cache, seqs, window=window), want), byte
    for bad in (np.nan, np.inf, -np.inf):
        x = q.clone()
        x[::3, 1] = bad
        got = S.kv4_attention(x, cache, seqs, window=window)
        rest = torch.ones(q.shape[:2], dtype=torch.bool, device=DEV)
        rest[::3, 1] = False
        assert torch.equal(got[rest], want[rest]), bad


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("new", [[1, 30], [3, 4], [5, 85]])
def test_attention_query_magnitudes(S, dtype, new):
    """Queries from 2^-100 to 2^60 within a row and between rows."""
    rng = np.random.default_rng(10)
    b = Batch(rng, new, [100, 90], 16)
    cache = random_cache(S, rng, b.pages, 2, 16, 64)
    q = rng.standard_normal((b.M, 4, 64))
    q[0] *= 2.0 ** rng.integers(-40, 0, (4, 64))
    q[1] *= 2.0 ** -100
    q[2] *= 2.0 ** 60
    q[3] = 0
    check_attention(S, dev(q.astype(np.float32), dtype), b, cache, scale=0.3)


def test_long_offsets(S):
    """A cache over 2^32 bytes: its last pages are written and read."""
    from w4a8_codebook_gemm_amd.attention import Sequences
    pages, H, P, D = 140000, 1, 256, 256
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)  # noqa: E731
    unit = torch.full((H,), 2.0 ** -14, device=DEV)
    cache = S.KV4Cache(z(pages, H, P, D // 2), z(pages, H, P, D // 2), z(pages, H, P, D // 16), z(pages, H, D // 16, P), unit, unit)
    small = S.KV4Cache.empty(4, H, P, D, DEV)
    rng = np.random.default_rng(11)
    x = dev(rng.standard_normal((300, H, D)).astype(np.float32))
    t = torch.arange(300, device=DEV)
    far, near = [(torch.where(t < P, a, b) * P + t % P) for a, b in ((pages - 1, pages - 3), (3, 1))]
    S.kv4_append(x, x, cache, far)
    S.kv4_append(x, x, small, near)
    q = dev(rng.standard_normal((300, 2, D)).astype(np.float32))
    for new in (1, 300):
        a, b = (S.kv4_attention(q[:new], c, Sequences(dev(np.array([tab], np.int32)), i32(0, new), i32(300)))
                for c, tab in ((cache, [pages - 1, pages - 3]), (small, [3, 1])))
        assert torch.equal(a, b)
    assert torch.equal(cache.k[pages - 1], small.k[3]) and torch.equal(cache.v_scale[pages - 3], small.v_scale[1])
    assert int(cache.k[:pages - 3].max()) == 0


class Far:
    """One sequence whose length is just below 2^31, nearly all of its pages given up, and the same sequence with
    `cut` positions (a multiple of every tile) taken from its front, where the operators must do the same."""

    def __init__(self, S, rng, new, page, hkv, d, held):
        from w4a8_codebook_gemm_amd.attention import Sequences
        self.width = 2 ** 31 // page - 1
        self.length = self.width * page - 1
        self.cut = 2 ** 31 - 4096
        self.pages = held + 2
        far = torch.full((1, self.width), -1, dtype=torch.int32, device=DEV)
        far[0, -held:] = dev(rng.permutation(self.pages)[:held].astype(np.int32))
        near = far[:, self.cut // page:].contiguous()
        self.seqs = [Sequences(t, i32(0, new), i32(n)) for t, n in ((far, self.length), (near, self.length - self.cut))]
        self.cache = random_cache(S, rng, self.pages, hkv, page, d)


@pytest.mark.parametrize("new,Hq,Hkv,D", [
    (1, 6, 1, 256), (1, 8, 2, 128), (1, 2, 2, 64),        # blocks of 16 rows
    (6, 8, 1, 128), (9, 4, 2, 256),                       # more of them
    (6, 256, 32, 128), (20, 64, 32, 64),                  # blocks of 32 rows
    (100, 2, 1, 256), (90, 4, 2, 128), (300, 3, 1, 64),   # the prompt kernel
])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [1, 1500])
def test_lengths_up_to_2_31_with_a_window(S, new, Hq, Hkv, D, dtype, window):
    rng = np.random.default_rng(new + D)
    f = Far(S, rng, new, 16, Hkv, D, held=100)
    q = dev(rng.standard_normal((new, Hq, D)).astype(np.float32), dtype)
    far, near = (S.kv4_attention(q, f.cache, s, window=window) for s in f.seqs)
    assert bool((near.abs().amax(-1) > 0).all()) and torch.equal(far, near)


@pytest.mark.parametrize("new,dtype", [([1, 1, 1, 1], BF), ([1, 3, 1, 2], F32), ([300, 20, 150, 1], BF)])
def test_attention_is_deterministic_and_leaves_its_workspace(S, new, dtype):
    rng = np.random.default_rng(12)
    b = Batch(rng, new, [3000, 700, 2000, 1500], 32)
    cache = random_cache(S, rng, b.pages, 2, 32, 128)
    q = dev(rng.standard_normal((b.M, 12, 128)).astype(np.float32), dtype)
    ws = S.kv4_attention_workspace(b.M, 4, 12, 2, 128, DEV)
    ws[S.COUNTER_BYTES:] = 255                            # may hold anything
    seqs = b.seqs()
    first = S.kv4_attention(q, cache, seqs, workspace=ws)
    for _ in range(5):
        assert torch.equal(S.kv4_attention(q, cache, seqs, workspace=ws), first)
    assert torch.equal(S.kv4_attention(q, cache, seqs), first)
    # the same workspace for another shape in between
    small = Batch(rng, [2], [50], 32)
    check_attention(S, q[:2], small, cache, workspace=ws)
    assert torch.equal(S.kv4_attention(q, cache, seqs, workspace=ws), first)


@pytest.mark.parametrize("M,B", [(1, 3), (500, 2), (300, 400)])
def test_batches_without_a_token_or_a_length(S, M, B):
    from w4a8_codebook_gemm_amd.attention import Sequences
    rng = np.random.default_rng(17)
    cache = random_cache(S, rng, 4, 8, 16, 64)
    zeros = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    table = torch.zeros(B, 2, dtype=torch.int32, device=DEV)
    q = torch.randn(M, 8, 64, device=DEV)
    out = torch.full_like(q, 5.0)
    S.kv4_attention(q, cache, Sequences(table, zeros, torch.full((B,), 20, dtype=torch.int32, device=DEV)), out=out)
    assert bool((out == 5.0).all())
    cu = torch.clamp(torch.arange(B + 1, device=DEV) * (-(-M // B)), max=M).to(torch.int32)
    S.kv4_attention(q, cache, Sequences(table, cu, zeros[:B].clone()), out=out)
    assert bool((out == 0).all())


def test_two_graphs_that_share_a_workspace(S):
    """Captured calls of quite different shapes on one workspace, replayed in turn with eager calls between."""
    rng = np.random.default_rng(16)
    cache = random_cache(S, rng, 400, 2, 32, 128)
    ws = S.kv4_attention_workspace(512, 4, 12, 2, 128, DEV)
    runs = []
    for new, lens, dtype in (([1, 1, 1], [3000, 700, 2100], BF), ([300, 40], [1500, 900], BF), ([4, 2], [2500, 30], F32)):
        b = Batch(rng, new, lens, 32)
        b.table = rng.integers(0, 400, b.table.shape).astype(np.int32)
        q, seqs = dev(rng.standard_normal((b.M, 12, 128)).astype(np.float32), dtype), b.seqs()
        runs.append((q, seqs, S.kv4_attention(q, cache, seqs), torch.empty_like(q)))
    torch.cuda.synchronize()
    graphs = []
    for q, seqs, _, out in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            S.kv4_attention(q, cache, seqs, workspace=ws, out=out)
        graphs.append(g)
    for turn in range(6):
        for i in rng.permutation(len(runs)):
            runs[i][3].fill_(3.0)
            graphs[i].replay()
            if turn % 2:
                q, seqs, want, _ = runs[(i + 1) % len(runs)]
                assert torch.equal(S.kv4_attention(q, cache, seqs, workspace=ws), want)
            assert torch.equal(runs[i][3], runs[i][2])


def test_streams_and_two_calls_at_once(S):
    """Calls on other streams than the default, with a workspace each, at the same time."""
    rng = np.random.default_rng(13)
    b = Batch(rng, [1, 1], [5000, 3000], 64)
    cache = random_cache(S, rng, b.pages, 2, 64, 256)
    seqs = b.seqs()
    qs = [dev(rng.standard_normal((2, 12, 256)).astype(np.float32), BF) for _ in range(2)]
    xs, r, w = [torch.randn(64, 512, device=DEV) for _ in range(2)], torch.randn(64, 512, device=DEV), torch.rand(512, device=DEV)
    want = [(S.kv4_attention(q, cache, seqs), S.add_norm_prepare(x, w, r)) for q, x in zip(qs, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = []
    for q, x, st in zip(qs, xs, streams):
        with torch.cuda.stream(st):
            ws = S.kv4_attention_workspace(2, 2, 12, 2, 256, DEV)
            got.append([(S.kv4_attention(q, cache, seqs, workspace=ws), S.add_norm_prepare(x, w, r)) for _ in range(4)])
    torch.cuda.synchronize()
    for outs, (o, p) in zip(got, want):
        for a, c in outs:
            assert torch.equal(a, o) and torch.equal(c.h, p.h) and torch.equal(c.x_q, p.x_q) and torch.equal(c.s_x, p.s_x)


@pytest.mark.parametrize("new", [[1, 3], [50, 70]])
def test_attention_scales_and_windows_at_their_limits(S, new):
    rng = np.random.default_rng(31)
    b = Batch(rng, new, [300, 90], 16)
    cache = random_cache(S, rng, b.pages, 2, 16, 64)
    q = dev(rng.standard_normal((b.M, 4, 64)).astype(np.float32), F32)
    for scale in (-0.2, 0.0, 1e-30):
        check_attention(S, q, b, cache, scale=scale)
    seqs = b.seqs()
    want = S.kv4_attention(q, cache, seqs)
    for window in (2 ** 40, 2 ** 31, 2 ** 31 - 1, 300):
        assert torch.equal(S.kv4_attention(q, cache, seqs, window=window), want)
    assert torch.equal(S.kv4_attention(-q, cache, seqs, scale=-(64 ** -0.5)), want)


def test_captured_calls_that_make_their_own_outputs_and_workspace(S):
    rng = np.random.default_rng(32)
    b = Batch(rng, [2, 90], [400, 700], 32)
    cache = random_cache(S, rng, b.pages, 2, 32, 128)
    q = dev(rng.standard_normal((b.M, 4, 128)).astype(np.float32), BF)
    x, r, w = torch.randn(9, 768, device=DEV), torch.randn(9, 768, device=DEV), torch.rand(768, device=DEV)
    p = make_pages(S, rng, [5, 40, 0], 20, 16, 50)
    pages, new = on_gpu(S, p, 16), i32(3, 200, 0)
    seqs = b.seqs()
    calls = lambda out: (S.kv4_attention(q, cache, seqs), *S.add_norm_prepare(x, w, r, normed_dtype=BF),  # noqa: E731
                         *vars(S.pages_assign(pages, new, 210, out=out)).values())
    tensors = lambda t: [y for y in t if isinstance(y, torch.Tensor)]  # noqa: E731
    want = [y.clone() for y in tensors(calls(S.Batch.empty(3, 210, DEV)))]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = tensors(calls(S.Batch.empty(3, 210, DEV)))
    for turn in range(5):
        for y in got:
            y.zero_()
        graph.replay()
        again = tensors(calls(S.Batch.empty(3, 210, DEV)))
        if turn % 2:
            torch.cuda.synchronize()
        assert len(got) == len(want) == 11
        for a, c, e in zip(got, want, again):
            assert torch.equal(a, c) and torch.equal(e, c)


# ----------------------------------------------------------------------------- together

def test_decoder_step_captured_and_replayed(S):
    """The whole run as a decoder's step uses it -- pages, norm, projections, rotation, append, attention,
    output projection, norm and the next product, drafts refused -- captured once and replayed, against
    the same calls made eagerly, the 64-bit attention and the layers' own activation preparation."""
    import w4a8_codebook_gemm_amd as w
    from w4a8_codebook_gemm_amd import attention as A
    torch.manual_seed(0)
    K, Hq, Hkv, D, P, B, T = 512, 4, 2, 128, 16, 3, 2
    M = B * T
    quant = lambda n, k, s: w.quantize_weight(torch.randn(n, k, device=DEV) / k ** 0.5, seed=s)  # noqa: E731
    wq, wk, wv, wo, wm = (quant(n, k, i) for i, (n, k) in enumerate([(Hq * D, K), (Hkv * D, K), (Hkv * D, K), (K, Hq * D), (256, K)]))
    freq, attn = A.rope_frequencies(64, 1e6, device=DEV)
    nw, n1, n2 = torch.randn(D, device=DEV) * 0.1, torch.rand(K, device=DEV), torch.rand(K, device=DEV)
    new = torch.full((B,), T, dtype=torch.int32, device=DEV)

    class Run:
        def __init__(self):
            self.pages = S.Pages.empty(B, 5, B * 5, P, DEV)
            self.batch = S.Batch.empty(B, M, DEV, self.pages.seq_lens, self.pages.free_count)
            self.cache = S.KV4Cache.empty(B * 5, Hkv, P, D, DEV)
            self.seqs = A.Sequences(self.pages.page_table, self.batch.cu_tokens, self.batch.seq_lens)
            self.x, self.h, self.refused = torch.zeros(M, K, device=DEV), torch.zeros(M, K, device=DEV, dtype=BF), i32(0, 1, 0)
            self.ws = S.kv4_attention_workspace(M, B, Hq, Hkv, D, DEV)

        def step(self):
            b = S.pages_assign(self.pages, new, M, out=self.batch)
            p = S.add_norm_prepare(self.x, n1, self.h, h_out=self.h, weight_offset=1.0, normed_dtype=F32)
            q, k, v = w.linear_multi(p.x_q, p.s_x, [wq, wk, wv])
            q, k = A.qk_norm_rope(q.view(M, Hq, D), k.view(M, Hkv, D), b.positions, freq, q_weight=nw, k_weight=nw,
                                  weight_offset=1.0, attn_factor=attn, out_dtype=F32)
            S.kv4_append(k, v.view(M, Hkv, D), self.cache, b.slots)
            o = S.kv4_attention(q, self.cache, self.seqs, workspace=self.ws)
            y = w.forward(o.view(M, Hq * D), wo)
            z = S.add_norm_prepare(y, n2, self.h, h_out=self.h, weight_offset=1.0)
            y = w.linear(z.x_q, z.s_x, wm)
            S.pages_release(self.pages, self.pages.seq_lens - self.refused)
            return q, o, p.normed, p.x_q, p.s_x, self.h, y

    eager, cap = Run(), Run()
    xs = [torch.randn(M, K, device=DEV) for _ in range(20)]
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
        assert torch.equal(eager.pages.seq_lens, cap.pages.seq_lens) and torch.equal(eager.pages.free_pages, cap.pages.free_pages)
        xq, sx = w.prepare_activation(want[2])
        assert torch.equal(xq, want[3]) and torch.equal(sx, want[4])
    assert eager.pages.seq_lens.tolist() == [40, 20, 40]
    b = Batch.__new__(Batch)
    # (as attention saw them, before one draft was refused)
    b.table, b.cu, b.lens = eager.pages.page_table.cpu().numpy(), eager.batch.cu_tokens.cpu().numpy(), np.array([40, 21, 40])
    check_attention(S, want[0], b, eager.cache, out=want[1])


def test_binding_refusals_on_the_gpu(S):
    from w4a8_codebook_gemm_amd.attention import Sequences
    rng = np.random.default_rng(14)
    cache = random_cache(S, rng, 4, 2, 16, 64)
    s = Sequences(dev(np.zeros((1, 2), np.int32)), i32(0, 2), i32(2))
    q = torch.randn(2, 4, 64, device=DEV)
    for bad in (q.half(), q.double()):
        with pytest.raises(TypeError):
            S.kv4_attention(bad, cache, s)
    for bad in (q.cpu(), q[:, :, :32], q.transpose(0, 1)):
        with pytest.raises(ValueError):
            S.kv4_attention(bad, cache, s)
    with pytest.raises(ValueError):
        S.kv4_attention(q, cache, s, out=torch.empty(2, 4, 32, device=DEV))
    for kw in (dict(window=3, causal=False), dict(window=-1), dict(scale=float("nan"))):
        with pytest.raises(S.ServingError):
            S.kv4_attention(q, cache, s, **kw)
    with pytest.raises(S.ServingError):
        S.kv4_attention(q[:, :3].contiguous(), cache, s)
    with pytest.raises(S.ServingError):
        S.kv4_attention(q, cache, s, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
    for window in ((1 << 64) + 3, 1 << 63):
        with pytest.raises(ValueError, match="window"):
            S.kv4_attention(q, cache, s, window=window)
    assert torch.equal(S.kv4_attention(q, cache, s, window=(1 << 63) - 1), S.kv4_attention(q, cache, s))
    k, slots = torch.randn(2, 2, 64, device=DEV), torch.arange(2, device=DEV)
    with pytest.raises(TypeError):
        S.kv4_append(k, k.bfloat16(), cache, slots)
    with pytest.raises(TypeError):
        S.kv4_append(k, k, cache, slots.int())
    for a, b, c in ((k, k[:1], slots), (k[:, :1], k, slots), (k, k, slots[:1]), (k, k, slots.cpu())):
        with pytest.raises(ValueError):
            S.kv4_append(a, b, cache, c)
    with pytest.raises(S.ServingError):
        S.kv4_append(k[:0], k[:0], cache, slots[:0])
    with pytest.raises(S.ServingError):                    # not 16-byte aligned
        S.kv4_append(k[:1], k[:1], cache, slots[1:])
    with pytest.raises(ValueError):
        S.KV4Cache(cache.k, cache.v, cache.k_scale, cache.v_scale.transpose(2, 3).contiguous(), cache.k_unit, cache.v_unit)
    with pytest.raises(TypeError):
        S.KV4Cache(cache.k, cache.v, cache.k_scale, cache.v_scale, cache.k_unit.double(), cache.v_unit)
    x, w = torch.randn(4, 512, device=DEV), torch.rand(512, device=DEV)
    for bad in (x.half(), x.double()):
        with pytest.raises(TypeError):
            S.add_norm_prepare(bad, w)
        with pytest.raises(TypeError):
            S.add_norm_prepare(x, w, bad)
    with pytest.raises(TypeError):
        S.add_norm_prepare(x, w.bfloat16())
    with pytest.raises(TypeError):
        S.add_norm_prepare(x, w, normed_dtype=torch.float16)
    for args, kw in (((x[0], w), {}), ((x, w[:256]), {}), ((x, w, x[:2]), {}), ((x.cpu(), w), {}), ((x, w.cpu()), {}),
                     ((x, w), dict(h_out=x)), ((x, w), dict(quantise=False)), ((x, w, x), dict(h_out=x.bfloat16())),
                     ((x.t().contiguous().t(), w), {})):
        with pytest.raises((ValueError, TypeError)):
            S.add_norm_prepare(*args, **kw)
    for a, kw in ((x[:, :320].contiguous(), {}), (x[:0], {}), (x[:, 1:257], {}), (x, dict(eps=-1.0)), (x, dict(eps=float("inf"))),
                  (x, dict(weight_offset=float("nan")))):
        with pytest.raises(S.ServingError):
            S.add_norm_prepare(a, w[:a.shape[1]], **kw)
    pages = S.Pages.empty(3, 4, 10, 16, DEV)
    with pytest.raises(TypeError):
        S.pages_assign(pages, torch.zeros(3, dtype=torch.int64, device=DEV), 3)
    for new in (i32(1, 1), i32(1, 1, 1).cpu()):
        with pytest.raises(ValueError):
            S.pages_assign(pages, new, 3)
    with pytest.raises(ValueError):
        S.pages_assign(pages, i32(1, 1, 1), 3, out=S.Batch.empty(3, 4, DEV))
    with pytest.raises(ValueError):
        S.pages_assign(pages, i32(1, 1, 1), 3, out=S.Batch.empty(2, 3, DEV))
    with pytest.raises(S.ServingError):
        S.pages_assign(pages, i32(1, 1, 1), 0)
    with pytest.raises(ValueError):
        S.pages_release(pages, i32(1, 1))
    with pytest.raises(S.ServingError):
        S.pages_release(S.Pages.empty(3, 4, 10, 24, DEV), i32(0, 0, 0))
    with pytest.raises(ValueError, match="page_size"):
        S.Pages.empty(3, 4, 10, (1 << 32) + 16, DEV)
    torch.cuda.synchronize()
