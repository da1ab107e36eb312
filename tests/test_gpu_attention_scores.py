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


@pytest.mark.parametrize("n", [1, 7, 100])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("power", [13, 20, 25.9])
def test_4_bit_cache(n, d, dtype, power):
    """Up to 2^20 the weight stands at 2^9 or more.  Below 2^26 the maximum lies 16 + 2 (its rounding) + 3 + 2 above the score, the
    argument's constant rounds by 2: 2^-11 or more, where an fp16 number has its 11 bits still and the sum of two is off by 2^-25.
    One number: 2^-11 of the weight; two: 2^-22, or 2^-25 / 2^-11.  Sums: 200 / 32 + 40 steps for numerator and denominator each, 70 for
    joining, of 2^-24: under 2^-16."""
    from w4a8_codebook_gemm_amd import serving as S
    import serving_ref as R
    k, v, q, score, table = case(d, n, dtype)
    cache = S.KV4Cache.empty(8, 1, 32, d, DEV)
    S.kv4_append(k, v, cache, torch.arange(LENGTH, device=DEV))
    kept = R.values4(*(t.cpu().numpy() for t in (cache.v, cache.v_scale.transpose(2, 3), cache.v_unit)))
    kept = torch.from_numpy(kept[:, 0].reshape(-1, 1, d)[:LENGTH]).to(DEV)
    seqs = S.Sequences(table, i32(0, n), i32(LENGTH))
    ratio = S.kv4_attention(q, cache, seqs, scale=2.0 ** power / score).double() / means(kept, n)
    weight = 2.0 ** -11 if dtype == BF else 2.0 ** -14 if power > 20 else 2.0 ** -22
    assert float((ratio - 1).abs().max()) < (weight + 2.0 ** -16 + torch.finfo(dtype).eps / 2) * 1.01
