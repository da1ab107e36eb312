"""The serving operators without a GPU: exports, argument validation (every status comes back before
any HIP call), the binding's own refusals, and the plain forms the GPU tests go by."""
import ctypes as C
import math
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

import serving_ref as R
from conftest import ROOT
from w4a8_codebook_gemm_amd import serving as S

FAKE, MIS = 0x10000, 0x10008


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(S.LIB_PATH):
        pytest.skip("library not built")
    return S.lib()


def test_exports_every_declared_symbol_and_nothing_else(L):
    text = open(os.path.join(ROOT, "include", "w4a8_serve.h")).read()
    names = re.findall(r"W4A8_API\s+[\w\s\*]+?\b(w4a8_\w+)\s*\(", text)
    assert sorted(names) == sorted(S.EXPORTS)
    out = os.popen(f"nm -D --defined-only {S.LIB_PATH}").read()
    assert sorted(x.split()[-1] for x in out.splitlines() if " T " in x) == sorted(names)


def test_status_strings(L):
    for s in range(8):
        assert L.w4a8_serve_status_string(s) not in (b"", b"unknown status")
    assert L.w4a8_serve_status_string(99) == b"unknown status"


def norm(L, **kw):
    v = dict(x=FAKE, xdt=0, xs=512, r=FAKE, rdt=1, rs=512, w=FAKE, off=1.0, eps=1e-6, M=3, K=512, h=FAKE, y=0, ydt=0, xq=FAKE,
             sx=FAKE) | kw
    return L.w4a8_add_norm_prepare(*v.values(), None)


def test_norm_validation(L):
    for kw in (dict(x=0), dict(w=0), dict(xq=0), dict(sx=0), dict(xq=0, sx=0), dict(r=0)):   # the last: h without r
        assert norm(L, **kw) == 1, kw
    for kw in (dict(M=0), dict(M=-1), dict(M=(1 << 24) + 1), dict(K=0), dict(K=128), dict(K=384), dict(K=65792, xs=65792, rs=65792),
               dict(K=-256), dict(xs=504), dict(xs=516), dict(rs=504), dict(rs=513), dict(xs=(1 << 31) + 8), dict(eps=-1.0),
               dict(eps=math.nan), dict(eps=math.inf), dict(off=math.inf), dict(off=math.nan)):
        assert norm(L, **kw) == 2, kw
    for kw in (dict(xdt=2), dict(rdt=-1), dict(y=FAKE, ydt=2)):
        assert norm(L, **kw) == 3, kw
    for kw in (dict(x=MIS), dict(r=MIS), dict(w=MIS), dict(h=MIS), dict(y=MIS), dict(xq=MIS), dict(sx=MIS)):
        assert norm(L, **kw) == 4, kw
    # what is not read is not looked at
    assert norm(L, r=0, h=0, rdt=9, rs=-5, x=MIS) == 4 and norm(L, ydt=9, x=MIS) == 4


def pages(**kw):
    v = dict(page_table=FAKE, seq_lens=FAKE, free_pages=FAKE, free_count=FAKE, B=2, table_width=4, num_pages=9, page_size=16) | kw
    return S.CPages(*v.values())


def batch(**kw):
    v = dict(cu_tokens=FAKE, seq_lens=FAKE, positions=FAKE, slots=FAKE, free_count=FAKE, missing=FAKE) | kw
    return S.CBatch(*v.values())


def assign(L, p=None, b=None, new=FAKE, M=5):
    p, b = p or pages(), b or batch()
    return L.w4a8_pages_assign(C.addressof(p), new, M, C.addressof(b), None)


def release(L, p=None, keep=FAKE, lens=FAKE, count=FAKE):
    p = p or pages()
    return L.w4a8_pages_release(C.addressof(p), keep, lens, count, None)


def test_pages_validation(L):
    for call in (assign, release):
        for name in ("page_table", "seq_lens", "free_pages", "free_count"):
            assert call(L, p=pages(**{name: 0})) == 1
            assert call(L, p=pages(**{name: MIS})) == 4
        for kw in (dict(B=0), dict(B=65537), dict(table_width=0), dict(table_width=(1 << 31) // 16), dict(num_pages=0),
                   dict(num_pages=1 << 31), dict(page_size=0), dict(page_size=8), dict(page_size=48), dict(page_size=512)):
            assert call(L, p=pages(**kw)) == 2, kw
    assert assign(L, new=0) == 1 and assign(L, new=MIS) == 4
    for M in (0, -1, (1 << 24) + 1):
        assert assign(L, M=M) == 2
    for name in ("cu_tokens", "seq_lens", "positions", "slots", "free_count", "missing"):
        assert assign(L, b=batch(**{name: 0})) == 1
        assert assign(L, b=batch(**{name: MIS})) == 4
    for name in ("keep", "lens", "count"):
        assert release(L, **{name: 0}) == 1 and release(L, **{name: MIS}) == 4
    assert L.w4a8_pages_assign(None, FAKE, 5, C.addressof(batch()), None) == 1
    assert L.w4a8_pages_assign(C.addressof(pages()), FAKE, 5, None, None) == 1
    assert L.w4a8_pages_release(None, FAKE, FAKE, FAKE, None) == 1


def cache(**kw):
    v = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, k_unit=FAKE, v_unit=FAKE, num_pages=8, kv_heads=4, page_size=64,
             head_dim=128) | kw
    return S.CKV4Cache(*v.values())


def seqs(**kw):
    from w4a8_codebook_gemm_amd.attention import CSequences
    v = dict(page_table=FAKE, cu_tokens=FAKE, seq_lens=FAKE, B=2, table_width=4) | kw
    return CSequences(*v.values())


def append(L, c=None, **kw):
    v = dict(k=FAKE, ks=512, v=FAKE, vs=512, dt=1, M=5) | {k: kw.pop(k) for k in list(kw) if k != "slots"}
    c = c or cache()
    return L.w4a8_kv4_append(*v.values(), C.addressof(c), kw.get("slots", FAKE), None)


def attn(L, c=None, s=None, **kw):
    v = dict(q=FAKE, qs=1024, dt=1, M=5, hq=8) | {k: kw.pop(k) for k in list(kw) if k in ("q", "qs", "dt", "M", "hq")}
    w = dict(scale=0.1, causal=1, window=0, o=FAKE, ws=FAKE, nb=1 << 40) | kw
    c, s = c or cache(), s or seqs()
    return L.w4a8_kv4_attention(*v.values(), C.addressof(c), C.addressof(s), *w.values(), None)


@pytest.mark.parametrize("call", [append, attn])
def test_cache_validation(L, call):
    for name in ("k", "v", "k_scale", "v_scale", "k_unit", "v_unit"):
        assert call(L, c=cache(**{name: 0})) == 1
        assert call(L, c=cache(**{name: MIS})) == 4
    for kw in (dict(num_pages=0), dict(num_pages=1 << 31), dict(kv_heads=0), dict(kv_heads=1025), dict(page_size=0),
               dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(head_dim=80), dict(head_dim=512)):
        assert call(L, c=cache(**kw)) == 2, kw
    assert call(L, dt=2) == 3


def test_append_validation(L):
    assert append(L, k=0) == 1 and append(L, v=0) == 1 and append(L, slots=0) == 1
    for kw in (dict(M=0), dict(M=(1 << 24) + 1), dict(ks=504), dict(vs=504), dict(ks=516), dict(vs=513)):
        assert append(L, **kw) == 2, kw
    wide = cache(kv_heads=1024, head_dim=256)      # more threads than a grid holds
    assert append(L, c=wide, ks=1 << 18, vs=1 << 18, M=1 << 17) == 2
    assert append(L, k=MIS) == 4 and append(L, v=MIS) == 4 and append(L, slots=MIS) == 4
    assert L.w4a8_kv4_append(FAKE, 512, FAKE, 512, 1, 5, None, FAKE, None) == 1


def test_attention_validation(L):
    assert attn(L, q=0) == 1 and attn(L, o=0) == 1
    for name in ("page_table", "cu_tokens", "seq_lens"):
        assert attn(L, s=seqs(**{name: 0})) == 1
        assert attn(L, s=seqs(**{name: MIS})) == 4
    for kw in (dict(B=0), dict(B=65537), dict(table_width=0), dict(table_width=(1 << 31) // 64)):
        assert attn(L, s=seqs(**kw)) == 2, kw
    for kw in (dict(M=0), dict(M=(1 << 24) + 1), dict(hq=0), dict(hq=6), dict(hq=8196), dict(qs=1016), dict(qs=1028),
               dict(causal=2), dict(window=-1), dict(window=5, causal=0), dict(scale=math.nan), dict(scale=math.inf),
               dict(hq=8192, qs=1 << 20, M=1 << 18)):
        assert attn(L, **kw) == 2, kw
    for kw in (dict(q=MIS), dict(o=MIS), dict(ws=MIS)):
        assert attn(L, **kw) == 4, kw
    ws = L.w4a8_kv4_attention_workspace_bytes
    for args in ((0, 1, 8, 4, 128), (1, 0, 8, 4, 128), (1, 1, 9, 4, 128), (1, 1, 8, 0, 128), (1, 1, 8, 4, 96), (1, 65537, 8, 4, 128)):
        assert ws(*args) == -2, args


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 512)
    with pytest.raises(ValueError, match="GPU"):
        S.add_norm_prepare(x, torch.zeros(512))
    with pytest.raises(ValueError, match="GPU"):
        S.KV4Cache.empty(2, 1, 16, 64, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        S.Pages.empty(2, 4, 8, 16, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        S.Batch.empty(2, 4, device="cpu")
    for far in (1 << 32, -(1 << 32), 1 << 64):
        for name in ("q_heads", "kv_heads", "head_dim"):
            with pytest.raises(ValueError, match=name):
                S.kv4_attention_workspace_bytes(**(dict(tokens=1, sequences=1, q_heads=8, kv_heads=4, head_dim=128) | {name: far}))


def test_import_needs_no_gpu_build_of_torch():
    """A torch built for CPUs lacks the accessors of streams and devices that calls on a GPU take."""
    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    hasattr(torch._C, n) and delattr(torch._C, n)\n"
            "from w4a8_codebook_gemm_amd import serving as S\n"
            "try:\n"
            "    S.add_norm_prepare(torch.zeros(2, 256), torch.zeros(256))\n"
            "except ValueError as e:\n"
            "    print('refused', e)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "must be on a GPU device" in r.stdout


def test_binding_raises_loudly_without_library(monkeypatch):
    monkeypatch.setattr(S, "_lib", None)
    monkeypatch.setattr(S, "LIB_PATH", "/nonexistent/libw4a8_serve.so")
    with pytest.raises(RuntimeError):
        S.lib()


def test_the_format_covers_its_range():
    """Every scale byte, steps that do not shrink, and the error of a value: half a step of the grid, and what the
    scale's five bits leave of the largest."""
    assert R.STEPS[0] == 0 and R.STEPS[255] == 507904 and np.all(np.diff(R.STEPS) > 0)
    rng = np.random.default_rng(0)
    unit = np.array([2.0 ** -14, 3e-5], np.float32)
    x = (rng.standard_normal((500, 2, 256)) * np.exp(rng.uniform(-3, 3, (500, 1, 1)))).astype(np.float32)
    codes, scales = R.quantise4(x, unit)
    back = R.values4(codes.transpose(1, 0, 2)[None], scales.transpose(1, 0, 2)[None], unit)[0].transpose(1, 0, 2)
    top = np.abs(x).reshape(500, 2, 16, 16).max(-1).repeat(16, -1)
    # a value above 4 of the 6 steps is off by one at most and by what is cut off a largest whose scale was
    # rounded down; one below 2 by a quarter
    assert np.all(np.abs(back - x) <= top / 6 * (1 + 2 ** -5) * np.where(np.abs(x) > 0.63 * top, 1.0, np.where(np.abs(x) > 0.31 * top, 0.5, 0.25)))
    rel = np.linalg.norm(back - x) / np.linalg.norm(x)
    assert 0.05 < rel < 0.12


def test_plain_pages_keep_every_page():
    """The plain forms undo each other and lose nothing, the list running out included."""
    rng = np.random.default_rng(1)
    table, lens, free, count = np.full((4, 6), -1), np.zeros(4, int), np.arange(15)[::-1].copy(), 15
    for _ in range(50):
        new = rng.integers(0, 30, 4)
        grown, cu, longer, positions, slots, left, missing = R.assign(table, lens, free, count, new, 16, int(new.sum()) + 1)
        back, same, n = R.release(grown, longer, free, left, lens, 16)
        assert n == count and np.array_equal(back[:n], free[:count]) and np.array_equal(same, lens)
        real = slots[slots >= 0]
        assert len(np.unique(real)) == len(real) and slots[-1] == -1
        keep = np.minimum(longer, rng.integers(0, 60, 4))
        free, lens, count = R.release(grown, longer, free, left, keep, 16)
        table = grown
        held = [table[b, e] for b in range(4) for e in range(-(-lens[b] // 16)) if table[b, e] >= 0]
        assert sorted(list(free[:count]) + held) == list(range(15))
