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
