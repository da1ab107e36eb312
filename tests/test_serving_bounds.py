"""What include/w4a8_serve.h says of how far values in 4 bits are off, on its plain form."""
import numpy as np
import pytest

import serving_ref as R

UNIT = np.float32(2.0 ** -14 * 1.37)
CUT = 3047424                                        # units: 6 sc(255)


def kept(x):
    """x [N, 16] in units of a head; the values kept, and each group's S, in units."""
    code, byte = R.quantise4((x * UNIT).astype(np.float32)[:, None], UNIT[None])
    v = R.values4(code[:, :, None], byte[:, :, None], UNIT[None])[:, 0, 0]
    return v / float(UNIT), R.STEPS[byte[:, 0, 0]]


def groups(rng, top):
    """16 values each, the first of them `top`, the others anywhere below it."""
    x = rng.uniform(-1, 1, (len(top), 16)) * top[:, None]
    x[:, 0] = top * rng.choice([-1, 1], len(top))
    return (x * UNIT).astype(np.float32).astype(np.float64) / float(UNIT)


def within(x, step):
    """S / 4 up to 2 S, S / 2 up to 4 S, S beyond; fp32 divisions move a border by 2^-23 of a value."""
    a = np.abs(x)
    return np.where(a <= 2 * step, step / 4, np.where(a <= 4 * step, step / 2, step)) + 2.0 ** -22 * a


@pytest.mark.parametrize("lo,hi", [(15.0001, 100.0), (90.0, CUT)])
def test_values_between_15_units_and_the_largest(lo, hi):
    rng = np.random.default_rng(1)
    x = groups(rng, np.exp(rng.uniform(np.log(lo), np.log(hi), 200000)))
    v, s = kept(x)
    assert np.all(np.abs(v - x) <= within(x, s[:, None]))
    big = np.abs(x).max(-1) >= 96
    t = np.abs(x).max(-1) / 6
    assert np.all(np.abs(s - t)[big] <= (2.0 ** -5 + 2.0 ** -22) * t[big])


def test_values_of_small_groups():
    """Up to 15 units: the same, or 3 units where that is more."""
    rng = np.random.default_rng(2)
    x = groups(rng, rng.uniform(0, 15, 200000))
    v, s = kept(x)
    err = np.abs(v - x)
    assert np.all(err <= np.maximum(within(x, s[:, None]), 3 * (1 + 2.0 ** -20)))
    assert err.max() > 2.9 and np.any(err > 1.4 * s[:, None])      # more than S: a group of 8.9 units is cut to 6


def test_values_beyond_the_largest_are_cut():
    rng = np.random.default_rng(3)
    x = groups(rng, CUT * np.exp(rng.uniform(0.001, 5, 20000)))
    v, s = kept(x)
    beyond = np.abs(x) > CUT
    assert np.all(s == R.STEPS[255]) and np.allclose(np.abs(v[beyond]), CUT, rtol=1e-6)
    assert np.all((np.abs(v - x) <= within(x, s[:, None]))[~beyond])
