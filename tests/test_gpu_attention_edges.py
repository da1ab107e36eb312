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
