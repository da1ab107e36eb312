"""The attention binding itself: its import, and numbers that do not fit the library's integers."""
import subprocess
import sys

import pytest
import torch

from conftest import ROOT
from w4a8_codebook_gemm_amd import attention as A


def test_import_needs_no_gpu_build_of_torch():
    """A torch built for CPUs lacks the accessors of streams and devices that calls on a GPU take."""
    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    hasattr(torch._C, n) and delattr(torch._C, n)\n"
            "from w4a8_codebook_gemm_amd import attention as A\n"
            "x = torch.zeros(2, 2, 64)\n"
            "try:\n"
            "    A.qk_norm_rope(x, None, torch.zeros(2, dtype=torch.int32), torch.zeros(8, dtype=torch.float64))\n"
            "except ValueError as e:\n"
            "    print('refused', e)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "must be on a GPU device" in r.stdout


@pytest.mark.gpu
def test_calls_run_with_torchs_public_accessors(monkeypatch):
    """What the private accessors give, the public ones give too."""
    x = torch.randn(5, 2, 64, device="cuda:0")
    pos = torch.arange(5, dtype=torch.int32, device="cuda:0")
    freq, _ = A.rope_frequencies(32, device="cuda:0")
    want, _ = A.qk_norm_rope(x, None, pos, freq)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert A._public_raw_stream(0) == side.cuda_stream == A._raw_stream(0)
    monkeypatch.setattr(A, "_raw_stream", A._public_raw_stream)
    monkeypatch.setattr(A, "_current_device", torch.cuda.current_device)
    got, _ = A.qk_norm_rope(x, None, pos, freq)
    assert torch.equal(got, want)


@pytest.mark.parametrize("far", [1 << 32, -(1 << 32), 1 << 64])
def test_numbers_past_the_librarys_integers_are_refused(far):
    """Their low bits alone would pass for a good call."""
    with pytest.raises(ValueError, match="does not fit"):
        A.rope_frequencies(far + 16, device="cpu")
    good = dict(tokens=1, sequences=1, q_heads=8, kv_heads=4, head_dim=128)
    for name in good:
        wrap = far if name in ("q_heads", "kv_heads", "head_dim") else 1 << 64
        with pytest.raises(ValueError, match=name):
            A.kv_attention_workspace_bytes(**good | {name: good[name] + wrap})


@pytest.mark.gpu
def test_windows_past_the_librarys_integers_are_refused():
    cache = A.KVCache.empty(2, 1, 16, 64, device="cuda:0")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda:0")  # noqa: E731
    s = A.Sequences(i32([0, 1]), i32(0, 2), i32(20))
    q = torch.randn(2, 2, 64, device="cuda:0")
    want = A.kv_attention(q, cache, s)
    assert torch.equal(A.kv_attention(q, cache, s, window=(1 << 63) - 1), want)
    for window in ((1 << 64) + 3, 1 << 63):
        with pytest.raises(ValueError, match="window"):
            A.kv_attention(q, cache, s, window=window)
    with pytest.raises(A.AttentionError):
        A.kv_attention(q, cache, s, window=-1)
