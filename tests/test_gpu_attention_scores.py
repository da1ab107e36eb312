"""Attention where scores are as large as include/w4a8_attn.h and include/w4a8_serve.h let them be.  All keys are alike, so all
positions weigh the same whatever the scores are: what is left of them are the exponents' roundings."""
import numpy as np
import pytest
import torch

from test_gpu_attention import A, BF, DEV, F32  # noqa: F401  (A is a fixture)

pytestmark = pytest.mark.gpu
LENGTH = 200


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def case(d, n, dtype):
    """LENGTH equal keys, positive values, n queries along the key; the score in powers of two at scale 1."""
    g = torch.Generator().manual_seed(d + n)
    k = torch.randn(1, 1, d, generator=g).expand(LENGTH, 1, d).contiguous().to(DEV)
    v = (torch.rand(LENGTH, 1, d, generator=g) + 0.5).to(DEV)
    q = k[:n].to(dtype)
    score = float((q[0].double() * k[0].double()).sum()) * 1.4426950408889634
    return k, v, q, score, torch.arange(8, dtype=torch.int32, device=DEV)[None]


def means(v, n):
    """The mean value that each of the last n positions sees, in 64 bits."""
    return (v.double().cumsum(0) / torch.arange(1, LENGTH + 1, device=DEV)[:, None, None])[LENGTH - n:]


@pytest.mark.parametrize("n", [1, 7, 100])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("power", [13, 20, 23.9])
def test_int8_cache(A, n, d, dtype, power):  # noqa: F811
    """Below 2^24 an exponent's argument rounds by half at the most: weights are within 2^0.5 of themselves, a row's mean of positive
    values within a factor of 2.  The output's half step (2^-8) and the cache's (1.5 / 254 of 0.5) are 2% at most."""
    k, v, q, score, table = case(d, n, dtype)
    cache = A.KVCache.empty(8, 1, 32, d)
    A.kv_append(k, v, cache, A.Sequences(table, i32(0, LENGTH), i32(LENGTH)))
    o = A.kv_attention(q, cache, A.Sequences(table, i32(0, n), i32(LENGTH)), scale=2.0 ** power / score).double()
    ratio = o / means(v, n)
    assert float(ratio.min()) > 0.49 and float(ratio.max()) < 2.04
