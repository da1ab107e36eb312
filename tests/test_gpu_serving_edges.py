"""The serving operators on the GPU where their arithmetic or their division of work is at its edge.  The plain forms,
batches and bounds are those of tests/test_gpu_serving.py but where a test states its own."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import test_gpu_serving as G
from test_gpu_serving import F32, S  # noqa: F401  (S is a fixture)

pytestmark = pytest.mark.gpu
DEV = G.DEV


# ----------------------------------------------------------------------------- the norm's factor

def rows_next_to_a_border(rng, count, away):
    """Rows of 256 whose factor 1 / sqrt(mean h^2) is `away` of itself beside a border between two fp32 numbers, and the
    number that it rounds to.  A few squares reach the sum that this wants; a last value of 2^-60, whose square the sum
    does not see, shows the factor itself in the norm."""
    rows, want = np.zeros((count, 256), np.float32), np.zeros(count, np.float32)
    for i in range(count):
        down = np.float32(rng.uniform(1, 4))
        up = np.nextafter(down, np.float32(8))
        border = (Fraction(float(down)) + Fraction(float(up))) / 2
        target = 256 / border ** 2 * (1 + (2 if i % 2 else -2) * Fraction(away))
        rest, at = target, 7 * (i % 5)
        for j in range(4):
            v = np.float32(np.sqrt(float(rest)))
            if Fraction(float(v)) ** 2 > rest:
                v = np.nextafter(v, np.float32(0))
            rows[i, at + 50 * j] = v
            rest -= Fraction(float(v)) ** 2
        total = sum(Fraction(float(v)) ** 2 for v in rows[i] if v)
        # the factor's distance from the border is half of the sum's
        off = abs(total * border ** 2 / 256 - 1) / 2
        assert Fraction(away) / 2 < off < 2 * Fraction(away)
        want[i] = up if total * border ** 2 < 256 else down
        rows[i, 255] = 2.0 ** -60
    return rows, want


def test_norm_factors_next_to_a_border(S):  # noqa: F811
    """2^-50.5 of themselves or more beside it.  Four squares in any order round the sum by at most 4 x 2^-53, so the factor by
    2 x 2^-53; the mean divides by a power of two; a root that is right to 2^-52 makes it 2^-51."""
    rows, want = rows_next_to_a_border(np.random.default_rng(20), 512, 2.0 ** -49.5)
    x = G.dev(rows)
    got = S.add_norm_prepare(x, torch.ones(256, device=DEV), eps=0.0, normed_dtype=F32, quantise=False).normed
    factor = got[:, 255].cpu().numpy() * np.float32(2.0 ** 60)
    assert int((factor != want).sum()) == 0


# ----------------------------------------------------------------------------- how attention for few rows cuts its work

def split_plan(new, lens, hq, hkv, d):
    """What k_kv4_split makes of a batch without a window: rows of a block, tiles of a workgroup's share (0: an even
    cut of the line), whether a unit's cost lies on the line, the most pieces of a unit, whether waves have whole units."""
    cu, group, waves = torch.cuda.get_device_properties(0).multi_processor_count, hq // hkv, 4
    rows, heads, wgs = -(-sum(new) * group // len(new)), len(new) * hkv, 2 * cu
    assert rows <= 64
    nb = 2 if d < 256 and rows > 16 and heads >= (cu // 8 if rows > 32 else cu // 2) else 1
    t = 32 * (256 // d)
    tiles = [max(1, -(-n // t)) for m, n in zip(new, lens) for _ in range(-(-m * group // (16 * nb)) * hkv)]
    solo = nb == 1 and d < 256 and heads >= wgs * waves and len(tiles) >= wgs * waves and \
        max(tiles) - sum(tiles) // len(tiles) <= len(tiles) // wgs
    line, c = sum(tiles), -(-sum(tiles) // (wgs * waves)) * waves
    while c <= 8 * waves:
        if sum(-(-x // c) for x in tiles) <= wgs:
            return 16 * nb, c, False, max(-(-x // c) for x in tiles), solo
        c += waves
    over = (10 if nb == 2 else 8) if nb == 1 or len(tiles) >= wgs else 0
    part = (line + over * len(tiles)) / wgs
    return 16 * nb, 0, over > 0, int(max(tiles) / part), solo


def shared_pages(rng, b, pages):
    """The batch on a cache of few pages, which its sequences share."""
    b.pages = pages
    b.table = rng.integers(0, pages, b.table.shape).astype(np.int32)


def attention64(q, cache, b):
    """Causal attention in 64 bits on the GPU, a sequence and cache head at a time, and what attention_ref.attention gives for
    its bounds."""
    M, hq, d = q.shape
    k, v = (G.dev(x) for x in G.dense(cache))
    P, hkv, g = k.shape[2], k.shape[1], hq // k.shape[1]
    o, A, T = (torch.zeros(M, hq, d, dtype=torch.float64, device=DEV) for _ in range(3))
    delta = torch.zeros(M, hq, 1, dtype=torch.float64, device=DEV)
    for i, n in enumerate(b.lens.tolist()):
        t = torch.arange(n, device=DEV)
        page, rows = G.dev(b.table[i])[t // P].long(), slice(int(b.cu[i]), int(b.cu[i + 1]))
        new = rows.stop - rows.start
        hidden = (t > n - new + torch.arange(new, device=DEV)[:, None]).repeat_interleave(g, 0)
        for h in range(hkv):
            kh, vh = k[page, h, t % P], v[page, h, t % P]
            heads = slice(h * g, (h + 1) * g)
            x = q[rows, heads].double().reshape(new * g, d)
            z = ((x @ kh.T.contiguous()) * d ** -0.5).masked_fill(hidden, -float("inf"))
            p = torch.softmax(z, -1)
            shape = (new, g, d)
            o[rows, heads], A[rows, heads] = (p @ vh).view(shape), (p @ vh.abs()).view(shape)
            T[rows, heads] = (p.amax(-1, keepdim=True) * ((~hidden).double() @ vh.abs())).view(shape)
            size = (x.abs() @ kh.abs().T.contiguous()).masked_fill(hidden, 0.0)
            delta[rows, heads] = (size.amax(-1) * d ** -0.5).view(new, g, 1)
    return [x.cpu().numpy() for x in (o, A, T, delta)]


def check_twice(S, q, b, cache):  # noqa: F811
    """Against the 64-bit form, and again to the bit; counters at zero after each call."""
    hkv, d = cache.k.shape[1], q.shape[2]
    ws = S.kv4_attention_workspace(b.M, len(b.lens), q.shape[1], hkv, d, DEV)
    ws[S.COUNTER_BYTES:] = 255
    seqs, outs = b.seqs(), []
    for _ in range(2):
        outs.append(S.kv4_attention(q, cache, seqs, workspace=ws))
        torch.cuda.synchronize()
        assert int(ws[:S.COUNTER_BYTES].max()) == 0
    assert torch.equal(*outs)
    ref, size, top, delta = attention64(q, cache, b)
    wide, length = q.dtype == F32, int(b.lens.max())
    e = ((d + 16) * G.U + (2.0 ** -22 if wide else 0)) * delta
    bound = (2 * e + 8 * G.U + 2 * (length / 32 + 40) * G.U + 70 * G.U + (2.0 ** -21 if wide else 2.0 ** -11)) * size
    # the row's largest weight stands at 2^10 or more, fp16's smallest numbers are 2^-24 apart
    bound = bound + 2.0 ** -35 * top + G.half_step(q.dtype) * (np.abs(ref) + bound)
    err = np.abs(G.f64(outs[0]) - ref)
    assert np.all(err <= bound), float((err / np.maximum(bound, 1e-300)).max())


@pytest.mark.parametrize("new,lo,hi,count,Hq,Hkv,D,page,behind", [
    (16, 10000, 20000, 8, 32, 8, 128, 32, False),        # fewer units than workgroups
    (16, 500, 4000, 32, 32, 8, 128, 16, True),           # as many or more: what a unit costs lies on the line
    (16, 16000, 30000, 8, 32, 8, 64, 64, False),
    (6, 2000, 8000, 64, 32, 8, 64, 16, True),
    (7, 300, 4000, 96, 18, 6, 128, 256, True),
])
@pytest.mark.parametrize("dtype", [G.BF, F32])
def test_blocks_of_32_rows_cut_anywhere(S, new, lo, hi, count, Hq, Hkv, D, page, behind, dtype):  # noqa: F811
    """Batches whose line is cut evenly, with pieces of units as they come (fewer than the 64 that the bound counts)."""
    rng = np.random.default_rng(new + count)
    lens = [int(x) for x in rng.integers(lo, hi, count)]
    block, share, over, pieces, _ = split_plan([new] * count, lens, Hq, Hkv, D)
    assert (block, share, over) == (32, 0, behind) and pieces > 0
    b = G.Batch(rng, [new] * count, lens, page)
    shared_pages(rng, b, 60)
    cache = G.random_cache(S, rng, b.pages, Hkv, page, D)
    q = G.dev(rng.standard_normal((b.M, Hq, D)).astype(np.float32), dtype)
    check_twice(S, q, b, cache)


@pytest.mark.parametrize("lens,Hq,Hkv,D,page,least", [
    ([40000], 24, 4, 256, 64, 65),
    ([131000], 6, 1, 256, 16, 500),                       # nearly every workgroup has a piece of it
    ([100000, 300], 8, 2, 64, 32, 65),
    ([70000], 6, 2, 128, 256, 65),
])
@pytest.mark.parametrize("dtype", [G.BF, F32])
def test_units_of_more_than_64_pieces(S, lens, Hq, Hkv, D, page, least, dtype):  # noqa: F811
    """Three levels of joining, 8 pieces at a node: 24 joins of three roundings, 72 u of A and not 70, while each piece's sum
    has lens / 32 / 64 steps at most where the bound counts lens / 32."""
    rng = np.random.default_rng(lens[0])
    assert split_plan([1] * len(lens), lens, Hq, Hkv, D)[3] >= least
    b = G.Batch(rng, [1] * len(lens), lens, page)
    shared_pages(rng, b, 100)
    cache = G.random_cache(S, rng, b.pages, Hkv, page, D)
    q = G.dev(rng.standard_normal((b.M, Hq, D)).astype(np.float32), dtype)
    check_twice(S, q, b, cache)


@pytest.mark.parametrize("new,length,Hq,Hkv,D,page", [(70, 70000, 5, 1, 256, 64), (90, 60000, 2, 1, 128, 16), (200, 100000, 2, 2, 64, 32)])
@pytest.mark.parametrize("dtype", [G.BF, F32])
def test_row_blocks_of_more_than_64_pieces(S, new, length, Hq, Hkv, D, page, dtype):  # noqa: F811
    """The prompt kernel's blocks of 256 rows (fp32 of 256: 128) and tiles of 8192 / D positions, cut for all compute units: two
    and two joined in 7 or 8 levels of three roundings, the rest as above."""
    cu = torch.cuda.get_device_properties(0).multi_processor_count
    blocks = -(-new * (Hq // Hkv) // (128 if D == 256 and dtype == F32 else 256)) * Hkv
    assert new * (Hq // Hkv) > 64 and cu // blocks > 64
    rng = np.random.default_rng(new)
    b = G.Batch(rng, [new], [length], page)
    shared_pages(rng, b, 100)
    cache = G.random_cache(S, rng, b.pages, Hkv, page, D)
    q = G.dev(rng.standard_normal((b.M, Hq, D)).astype(np.float32), dtype)
    check_twice(S, q, b, cache)


# ----------------------------------------------------------------------------- pages of wide tables

@pytest.mark.parametrize("B,width", [(3, 2 ** 20 + 1), (1030, 2 ** 20 + 1), (40, 2 ** 25), (11, 2 ** 27 - 1)])
def test_release_from_wide_tables(S, B, width):  # noqa: F811
    """Tables of so many entries that fewer than 1024 sequences go at a time: 1023, 32 and 8 of them."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 400, B)
    lens[::4] = width * 16 - rng.integers(0, 400, len(lens[::4]))
    keep = np.maximum(lens - rng.integers(-20, 200, B), 0)
    total, table, free = 30000, torch.empty((B, width), dtype=torch.int32, device=DEV), []
    at, seqs, entries = iter(rng.permutation(total)), [], []
    for b in reversed(range(B)):
        for e in reversed(range(-(-min(keep[b], lens[b]) // 16), -(-lens[b] // 16))):
            seqs.append(b)
            entries.append(e)
            free.append(next(at))
    table[torch.tensor(seqs, device=DEV), torch.tensor(entries, device=DEV)] = G.dev(np.array(free, np.int32))
    pages = S.Pages(table, G.dev(lens.astype(np.int32)), torch.full((total,), -9, dtype=torch.int32, device=DEV), G.i32(2), 16)
    got, count = S.pages_release(pages, G.dev(keep.astype(np.int32)))
    assert np.array_equal(got.cpu().numpy(), np.minimum(keep, lens)) and int(count) == 2 + len(free)
    assert pages.free_pages[:2 + len(free)].tolist() == [-9, -9] + [int(x) for x in free]
    assert bool((pages.free_pages[2 + len(free):] == -9).all())
