"""The 4-bit write's rotation (csrc/kv_cache_fp4.cu), checked on the CPU
through a model of its arithmetic, operation by operation in IEEE fp32: how
far its sines, cosines and angles are from the exact ones, which is what the
kernel's comment and the header state.

Bound of a sine or cosine.  Beside the table's exact hi + lo, the largest term
is cos a (cos delta - 1), |delta| <= pi / 256 (and the same of sin a): at most
c = (pi / 256)^2 / 2 < 2^-13.69.  Its factor cm takes three roundings (delta's
square, the bracket, the product), then product, sum and sum round once each,
every one by at most 2^-24 of c for the first three (the bracket lies just
below 1/2) and by half an fp32 unit of a value below 2^-13, 2^-38, for the rest:
3 * 2^-37.69 + 3 * 2^-38 < 2^-35.4; all else is below 2^-44."""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest

F = np.float32
BOUND = 2.0 ** -35.4


def _fma(a, b, c):
    """fp32 fma: the fp64 product of two fp32 is exact; the fp64 sum is rounded
    to odd, so that the second rounding is the only one that counts."""
    p, c = a.astype(np.float64) * np.asarray(b, np.float64), np.asarray(c, np.float64) + np.zeros(a.shape)
    s = p + c
    t = s - p
    e = (p - (s - t)) + (c - t)
    bits = s.view(np.int64)
    step = np.where((e > 0) == (s > 0), 1, -1)
    return np.where((e != 0) & (bits & 1 == 0), bits + step, bits).view(np.float64).astype(F)


def _two_sum(a, b):
    hi = a + b
    t = hi - a
    return hi, (a - (hi - t)) + (b - t)


def _two_prod(a, b):
    p = a * b
    return p, _fma(a, b, -p)


def _turn_radians():
    return np.longdouble(2) * (np.longdouble(math.pi) + np.longdouble("1.2246467991473531772e-16"))


def _table(k):
    """cos hi, cos lo, sin hi, sin lo of 2 pi k / 256."""
    if np.finfo(np.longdouble).nmant <= 52:
        pytest.skip("long double is no wider than double here")
    x = _turn_radians() * k.astype(np.longdouble) / 256
    out = []
    for v in (np.cos(x), np.sin(x)):
        hi = v.astype(F)
        out += [hi, (v - hi).astype(F)]
    return out


def _cos_sin_turn(turn):
    """The kernel's cos_sin_turn of uint64 fractions of a turn."""
    up = turn + np.uint64(1 << 55)
    ax, ay, az, aw = _table(up >> np.uint64(56))
    hi = (((up >> np.uint64(24)) & np.uint64(0xFFFFFFFF)).astype(np.uint32) ^ np.uint32(0x80000000))
    lo = (up & np.uint64(0xFFFFFF)).astype(np.uint32)
    r1 = (hi.view(np.int32) >> 12).astype(F)
    r2 = (((hi & np.uint32(0xFFF)) << np.uint32(10)) | (lo >> np.uint32(14))).astype(F)
    rs = r2 * F(2.0 ** -22)
    rh = r1 + rs
    rl = rs - (rh - r1)
    pi_hi = F(2 * math.pi * 2.0 ** -28)
    pi_lo = F(2 * math.pi * 2.0 ** -28 - float(pi_hi))
    dh, de = _two_prod(rh, pi_hi)
    dl = de + _fma(rh, pi_lo, rl * pi_hi)
    d2 = dh * dh
    sl = _fma(dh * d2, _fma(d2, F(1 / 120), F(-1 / 6)), dl)
    cm = _fma(d2, _fma(d2, F(1 / 24), F(-0.5)), -dh * dl)
    p, pe = _two_prod(-az, dh)
    h, l = _two_sum(ax, p)
    c = _two_sum(h, l + (_fma(ax, cm, pe) + (ay - _fma(az, sl, aw * dh))))
    p, pe = _two_prod(ax, dh)
    h, l = _two_sum(az, p)
    s = _two_sum(h, l + (_fma(az, cm, pe) + (aw + _fma(ax, sl, ay * dh))))
    return c, s


def _exact(turn):
    x = turn.astype(np.longdouble) / np.longdouble(2.0 ** 64)
    x = np.where(x > 0.5, x - 1, x) * _turn_radians()
    return np.cos(x), np.sin(x)


@pytest.mark.parametrize("seed", range(4))
def test_sines_and_cosines_within_the_stated_bound(seed):
    rng = np.random.default_rng(seed)
    turn = rng.integers(0, 2 ** 64, 1 << 18, dtype=np.uint64)
    if seed == 1:                                  # beside the table's borders, where delta is largest
        turn = (turn & np.uint64(0xFF00000000FFFFFF)) + np.uint64(1 << 55)
    if seed == 2:                                  # small angles
        turn >>= np.uint64(8) * (turn & np.uint64(7))
    worst = 0.0
    for (hi, lo), ref in zip(_cos_sin_turn(turn), _exact(turn)):
        err = np.abs((hi.astype(np.longdouble) - ref) + lo)
        worst = max(worst, float(err.max()))
    assert worst <= BOUND, math.log2(worst)
    if seed == 1:
        assert worst > 2.0 ** -38                  # the bound is not far from what happens


@pytest.mark.parametrize("bf16", [False, True])
def test_rotated_values_within_the_stated_bound(bf16):
    """u cos - w sin before its roundings: sqrt(2) 2^-35.4 of the pair's length
    from the sine and cosine, and sums of terms 2^-16 below it: under 2^-34."""
    rng = np.random.default_rng(5)
    n = 1 << 16
    turn = rng.integers(0, 2 ** 64, n, dtype=np.uint64)
    u, w = ((rng.standard_normal(n) * 2.0 ** rng.integers(-20, 20, n)).astype(F) for _ in range(2))
    if bf16:
        u, w = ((x.view(np.uint32) & np.uint32(0xFFFF0000)).view(F) for x in (u, w))
    (ch, cl), (sh, sl) = _cos_sin_turn(turn)
    if bf16:                                       # 16 leading bits: exact products
        cut = [(x.view(np.uint32) & np.uint32(0xFFFFFF00)).view(F) for x in (ch, sh)]
        cl, sl, ch, sh = (ch - cut[0]) + cl, (sh - cut[1]) + sl, cut[0], cut[1]
        assert (u.astype(float) * ch == (u * ch).astype(float)).all()
        s, se = _two_sum(u * ch, w * -sh)
        rest = se + _fma(u, cl, w * -sl)
    else:
        (p, pe), (q, qe) = _two_prod(u, ch), _two_prod(w, -sh)
        s, se = _two_sum(p, q)
        rest = se + (_fma(u, cl, pe) + _fma(w, -sl, qe))
    c, t = _exact(turn)
    err = np.abs((s.astype(np.longdouble) - (u * c - w * t)) + rest)
    assert (err <= np.hypot(u.astype(float), w.astype(float)) * 2.0 ** -34).all()


@pytest.mark.parametrize("theta", [1e4, 5e5, 1e6, 10.0, 0.5])
@pytest.mark.parametrize("d", [64, 128])
def test_angles_within_2_to_the_minus_50_of_themselves(theta, d):
    """The host's fractions of a turn per position (two powers, their product,
    a quotient: five roundings of half to one fp64 unit, below 2^-50 together)
    and 2^-64 from their truncation, against 60 digits."""
    getcontext().prec = 60
    pi2 = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    fine = [math.pow(theta, -2.0 * k / d) for k in range(8)]
    for j in range(d // 16):
        coarse = math.pow(theta, -16.0 * j / d)
        for k in range(8):
            x = coarse * fine[k] / (2 * math.pi)
            turn = int(math.ldexp(x - math.floor(x), 64))
            exact = (Decimal(theta).ln() * Decimal(-2 * (8 * j + k)) / Decimal(d)).exp() / pi2
            got = Decimal(turn) / Decimal(2 ** 64) + Decimal(math.floor(x))
            assert abs(got - exact) <= exact * Decimal(2) ** -50 + Decimal(2) ** -64
