"""The 8-bit scale rule at its borders: fl(m / 127) against the scale so far,
from exact rationals on the CPU, and the kernel's codes and scales there."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import int8


def nearest_f32(x):
    """A positive rational rounded to fp32, halves to even, by its definition (normal numbers)."""
    e = x.numerator.bit_length() - x.denominator.bit_length()
    while Fraction(2) ** e > x:
        e -= 1
    while Fraction(2) ** (e + 1) <= x:
        e += 1
    ulp = Fraction(2) ** (e - 23)
    n = x / ulp
    down = n.numerator // n.denominator
    rest = n - down
    if rest > Fraction(1, 2) or (rest == Fraction(1, 2) and down % 2):
        down += 1
    return np.float32(float(down * ulp))


def at_the_border(old, steps):
    """The float32 magnitudes `steps` steps around 127 * old."""
    m = np.array([old * np.float32(127)], np.float32)
    return (m.view(np.int32)[0] + np.asarray(steps)).astype(np.int32).view(np.float32)


def test_new_scale_at_its_borders():
    rng = np.random.default_rng(5)
    olds = np.concatenate([[0.01, 1 / 127, 1.0, 2.0 ** -100, 2.0 ** 100], rng.lognormal(0, 4, 300)]).astype(np.float32)
    stays = grows = 0
    for old in olds:
        for m in at_the_border(old, range(-6, 7)):
            want = nearest_f32(Fraction(float(m)) / 127)
            expect = old if want <= old else max(want, np.float32(2) * old)
            assert int8.new_scale(float(m), old) == expect, (m, old)
            stays, grows = stays + (want <= old), grows + (want > old)
    assert stays > 1000 and grows > 1000
    assert int8.new_scale(1.27, np.float32(0.01)) == np.float32(0.01)   # fl(1.27) / 127 is below fl(0.01)'s next number
    assert int8.new_scale(float(at_the_border(np.float32(0.01), 3)), np.float32(0.01)) == np.float32(0.02)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_the_kernel_at_the_borders(d):
    """Tokens appended to blocks whose scale is a few steps of m off: scales and codes bit for bit."""
    import torch

    from tests.helpers import ensure_built
    pk = ensure_built()
    rng = np.random.default_rng(d)
    H, nb = 13, 64
    pool = rng.integers(1, 256, (nb, H, 32 * d + 16), dtype=np.uint8)
    sc = rng.lognormal(0, 4, (nb, 1, 2)).astype(np.float32) * np.ones((1, H, 1), np.float32)
    pool[:, :, -16:-8] = sc.view(np.uint8)
    x = rng.uniform(-0.9, 0.9, (nb, H, d)) * (sc[:, :, :1] * 127)
    x = x.astype(np.float32)
    for b in range(nb):
        x[b, np.arange(H), rng.integers(0, d, H)] = at_the_border(sc[b, 0, 0], np.arange(H) - 6) * rng.choice([-1, 1], H)
    v = (x.astype(np.float64) / sc[:, :, :1] * sc[:, :, 1:]).astype(np.float32)
    slots = (np.arange(nb) * 16 + rng.integers(1, 16, nb)).astype(np.int64)
    want = pool.copy()
    int8.write_rows(x.astype(np.float64), slots, want, 0, d)
    int8.write_rows(v.astype(np.float64), slots, want, 1, d)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    got = dev(pool)
    pk.photon_kv_cache_write_int8(dev(x), dev(v), dev(np.zeros(nb, np.int32)), dev(slots), got, 1e4, "none")
    assert np.array_equal(got.cpu().numpy(), want)
    grown = int8.scales(want)[..., 0] > sc[..., 0]
    assert grown.any() and not grown.all()
