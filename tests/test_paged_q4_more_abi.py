"""Further CPU checks of the cache in 4 bits (include/paged_q4.h): its oracle."""
import numpy as np

from oracle import paged_q4 as O


def held(x):
    """What a cache holds of x [n, 16]."""
    return O.values(*O.quantise(x)).reshape(x.shape)


def test_oracle_errors_are_bounded_at_every_size():
    """With a group's largest a and its scale s: |x| <= 6 s is off by at most s, half the widest gap; beyond, x is cut off, by
    at most a - 6 s.  From a = 6 * 2^-6 on, s is within 1/16 of a / 6: max(s, a - 6 s) <= (1 + 1/16) a / 6.  Below, E4M3's
    numbers are 2^-9 apart, so s is within 2^-10 of a / 6, or 2^-9 where that is more: s <= a / 6 + 2^-10, or 2^-9, and
    a - 6 s <= 6 * 2^-10."""
    rng = np.random.default_rng(3)
    a = np.exp2(rng.uniform(-14, np.log2(2687), 500))
    a[:60] = (np.arange(60) % 20 + 0.5) * 6 * 2.0 ** -9 * np.repeat([1 - 1e-9, 1.0, 1 + 1e-9], 20)  # scales' borders
    x = rng.uniform(-1, 1, (500, 16)) * a[:, None]
    x[:, 0] = a
    x[:, 1:8] = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) / 6 * a[:, None]
    err = np.abs(held(x) - x).max(-1)
    bound = np.where(a >= 6 * 2.0 ** -6, (1 + 1 / 16) * a / 6, np.maximum(a / 6 + 2.0 ** -10, 3 * 2.0 ** -9))
    assert np.all(err <= bound * (1 + 1e-12))
    small = a < 0.03
    assert np.any(err[small] > 1.5 * (1 + 1 / 16) * a[small] / 6)   # (more than above that size)


def test_oracle_holds_the_smallest_as_zeros():
    x = np.full((1, 16), 2.0 ** -11)
    assert not held(x).any() and held(x * 1.001).all()
