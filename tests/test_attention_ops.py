"""The attention operators without a GPU: exports, argument validation (every status comes back
before any HIP call), the binding's own refusals and the rotary frequencies."""
import ctypes as C
import math
import os
import re

import numpy as np
import pytest
import torch

from conftest import ROOT
from w4a8_codebook_gemm_amd import attention as A

FAKE, MIS = 0x10000, 0x10008


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(A.LIB_PATH):
        pytest.skip("library not built")
    return A.lib()


def test_exports_every_declared_symbol_and_nothing_else(L):
    text = open(os.path.join(ROOT, "include", "w4a8_attn.h")).read()
    names = re.findall(r"W4A8_API\s+[\w\s\*]+?\b(w4a8_\w+)\s*\(", text)
    assert sorted(names) == sorted(A.EXPORTS)
    out = os.popen(f"nm -D --defined-only {A.LIB_PATH}").read()
    assert sorted(x.split()[-1] for x in out.splitlines() if " T " in x) == sorted(names)


def test_status_strings(L):
    for s in range(8):
        assert L.w4a8_attn_status_string(s) not in (b"", b"unknown status")
    assert L.w4a8_attn_status_string(99) == b"unknown status"


def heads(**kw):
    v = dict(x=FAKE, token_stride=1024, head_stride=256, heads=4, weight=FAKE, out=FAKE) | kw
    return A.CHeads(*v.values())


def rope(L, q=None, k=None, null_q=False, **kw):
    v = dict(M=3, d=256, xdt=0, odt=1, pos=FAKE, freq=FAKE, r=64, inter=0, factor=1.0, eps=1e-6, offset=0.0) | kw
    q = q or heads()
    return L.w4a8_qk_norm_rope(None if null_q else C.addressof(q), C.addressof(k) if k else None, *v.values(), None)


def test_rope_validation(L):
    assert rope(L, null_q=True) == 1
    for kw in (dict(pos=0), dict(freq=0)):
        assert rope(L, **kw) == 1
    for h in (heads(x=0), heads(out=0)):
        assert rope(L, q=h) == 1 and rope(L, k=h) == 1
    for kw in (dict(M=0), dict(M=-1), dict(M=(1 << 24) + 1), dict(d=96), dict(d=0), dict(r=0), dict(r=8), dict(r=24),
               dict(r=272), dict(inter=2), dict(eps=-1.0), dict(eps=math.nan)):
        assert rope(L, **kw) == 2, kw
    for h in (heads(heads=0), heads(head_stride=248), heads(head_stride=260), heads(token_stride=1028),
              heads(token_stride=-8), heads(heads=65537)):
        assert rope(L, q=h) == 2 and rope(L, k=h) == 2
    assert rope(L, q=heads(heads=256), M=1 << 23) == 2     # M * heads
    assert rope(L, xdt=2) == 3 and rope(L, odt=-1) == 3
    for kw in (dict(pos=MIS), dict(freq=MIS)):
        assert rope(L, **kw) == 4
    for h in (heads(x=MIS), heads(out=MIS), heads(weight=MIS)):
        assert rope(L, q=h) == 4 and rope(L, k=h) == 4


def cache(**kw):
    v = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, num_pages=8, kv_heads=4, page_size=64, head_dim=128) | kw
    return A.CCache(*v.values())


def seqs(**kw):
    v = dict(page_table=FAKE, cu_tokens=FAKE, seq_lens=FAKE, B=2, table_width=4) | kw
    return A.CSequences(*v.values())


def append(L, c=None, s=None, **kw):
    v = dict(k=FAKE, ks=512, v=FAKE, vs=512, dt=1, M=5) | kw
    c, s = c or cache(), s or seqs()
    return L.w4a8_kv_append(*v.values(), C.addressof(c), C.addressof(s), None)


def attn(L, c=None, s=None, **kw):
    v = dict(q=FAKE, qs=1024, dt=1, M=5, hq=8) | {k: kw.pop(k) for k in list(kw) if k in ("q", "qs", "dt", "M", "hq")}
    w = dict(scale=0.1, causal=1, window=0, o=FAKE, ws=FAKE, nb=1 << 40) | kw
    c, s = c or cache(), s or seqs()
    return L.w4a8_kv_attention(*v.values(), C.addressof(c), C.addressof(s), *w.values(), None)


BAD_CACHES = [dict(num_pages=0), dict(num_pages=1 << 31), dict(kv_heads=0), dict(kv_heads=1025), dict(page_size=0),
              dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(head_dim=80), dict(head_dim=512)]
BAD_SEQS = [dict(B=0), dict(B=65537), dict(table_width=0), dict(table_width=(1 << 31) // 64)]


@pytest.mark.parametrize("call", [append, attn])
def test_cache_and_sequences_validation(L, call):
    for name in ("k", "v", "k_scale", "v_scale"):
        assert call(L, c=cache(**{name: 0})) == 1
        assert call(L, c=cache(**{name: MIS})) == 4
    for name in ("page_table", "cu_tokens", "seq_lens"):
        assert call(L, s=seqs(**{name: 0})) == 1
        assert call(L, s=seqs(**{name: MIS})) == 4
    for kw in BAD_CACHES:
        assert call(L, c=cache(**kw)) == 2, kw
    for kw in BAD_SEQS:
        assert call(L, s=seqs(**kw)) == 2, kw
    assert call(L, dt=2) == 3


def test_append_validation(L):
    assert append(L, k=0) == 1 and append(L, v=0) == 1
    for kw in (dict(M=0), dict(M=(1 << 24) + 1), dict(ks=504), dict(vs=504), dict(ks=516), dict(vs=513)):
        assert append(L, **kw) == 2, kw
    assert append(L, k=MIS) == 4 and append(L, v=MIS) == 4
    assert L.w4a8_kv_append(FAKE, 512, FAKE, 512, 1, 5, None, None, None) == 1


def test_attention_validation(L):
    assert attn(L, q=0) == 1 and attn(L, o=0) == 1
    for kw in (dict(M=0), dict(M=(1 << 24) + 1), dict(hq=0), dict(hq=6), dict(hq=8196), dict(qs=1016), dict(qs=1028),
               dict(causal=2), dict(window=-1), dict(window=5, causal=0), dict(scale=math.nan), dict(scale=math.inf)):
        assert attn(L, **kw) == 2, kw
    assert attn(L, M=1 << 24, hq=256, qs=1 << 20) == 2      # M * q_heads
    for name in ("q", "o", "ws"):
        assert attn(L, **{name: MIS}) == 4
    f = L.w4a8_kv_attention_workspace_bytes
    for bad in [(0, 1, 8, 4, 128), (1, 0, 8, 4, 128), (1, 1, 8, 3, 128), (1, 1, 8, 4, 100), (1, 65537, 8, 4, 128)]:
        assert f(*bad) == -2, bad


def test_binding_refuses_what_the_library_cannot_see():
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        A.qk_norm_rope(x, None, torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.float64))
    with pytest.raises(ValueError):
        A.qk_norm_rope(torch.zeros(4, 64), None, torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.float64))
    with pytest.raises(ValueError):
        A.KVCache.empty(2, 2, 16, 64, device="cpu")
    with pytest.raises(ValueError):
        A.Sequences(torch.zeros(1, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        A.KVCache(x, x, x, x)


def test_binding_raises_loudly_without_library(monkeypatch):
    monkeypatch.setattr(A, "_lib", None)
    monkeypatch.setattr(A, "LIB_PATH", "/nonexistent/libw4a8_attn.so")
    with pytest.raises(RuntimeError):
        A.lib()


def test_rope_frequencies(L):
    r, base, factor, ctx = 64, 1e6, 8.0, 32768.0
    i = np.arange(r // 2)
    f = base ** (-2 * i / r)
    get = lambda *a, **kw: A.rope_frequencies(*a, device="cpu", **kw)  # noqa: E731
    tol = dict(rtol=1e-13, atol=0)   # a few roundings of pow
    t, a = get(r, base)
    np.testing.assert_allclose(t.numpy(), f, **tol)
    assert t.dtype == torch.float64 and t.shape == (32,) and a == 1.0
    t, a = get(r, base, "linear", factor)
    np.testing.assert_allclose(t.numpy(), f / factor, **tol)
    assert a == 1.0
    t, a = get(r, base, "ntk", factor)
    # the stretched base leaves the fastest pair as it is and slows the slowest by the factor
    np.testing.assert_allclose([t[0], t[-1]], [1.0, f[-1] / factor], rtol=1e-12)
    t, a = get(r, base, "yarn", factor, ctx)
    assert a == np.float32(0.1 * math.log(factor) + 1)
    turns = ctx * f / (2 * math.pi)
    assert np.allclose(t.numpy()[turns > 40], f[turns > 40], **tol)
    assert np.allclose(t.numpy()[turns < 0.6], f[turns < 0.6] / factor, **tol)
    mid = t.numpy()[(turns < 25) & (turns > 1.5)] / f[(turns < 25) & (turns > 1.5)]
    assert len(mid) and np.all(np.diff(mid) < 0) and np.all(mid < 1) and np.all(mid > 1 / factor)
    t, _ = get(2, base, "yarn", factor, 3.0)     # a ramp without width
    assert np.all(np.isfinite(t.numpy()))


@pytest.mark.parametrize("args,status", [
    ((0, 1e4, 0), 2), ((3, 1e4, 0), 2), ((-4, 1e4, 0), 2), ((16, 1.0, 0), 2), ((16, math.nan, 0), 2), ((16, math.inf, 0), 2),
    ((16, 1e4, 4), 3), ((16, 1e4, -1), 3), ((16, 1e4, 1, 0.5), 2), ((16, 1e4, 1, math.nan), 2), ((2, 1e4, 2, 2.0), 2),
    ((16, 1e4, 3, 2.0, 0.0), 2), ((16, 1e4, 3, 2.0, 100.0, 1.0, 1.0), 2), ((16, 1e4, 3, 2.0, 100.0, 1.0, 0.0), 2)])
def test_rope_frequencies_refusals(L, args, status):
    full = list(args) + [1.0, 1.0, 32.0, 1.0][len(args) - 3:]
    buf, a = (C.c_double * 64)(), C.c_float()
    assert L.w4a8_rope_frequencies(*full, C.addressof(buf), C.addressof(a)) == status


def test_rope_frequencies_null(L):
    buf, a = (C.c_double * 64)(), C.c_float()
    assert L.w4a8_rope_frequencies(16, 1e4, 0, 1.0, 1.0, 32.0, 1.0, None, C.addressof(a)) == 1
    assert L.w4a8_rope_frequencies(16, 1e4, 0, 1.0, 1.0, 32.0, 1.0, C.addressof(buf), None) == 1
    with pytest.raises(ValueError):
        A.rope_frequencies(16, scaling="other", device="cpu")
    with pytest.raises(A.AttentionError):
        A.rope_frequencies(15, device="cpu")
