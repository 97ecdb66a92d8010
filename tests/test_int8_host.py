"""8-bit cache and q/k norms without a GPU: the record layout and the oracle's
definitions pinned, and the refusals of the C entry points before any launch."""
import ctypes

import numpy as np
import pytest

import oracle
from oracle import int8
from tests.helpers import ensure_built


@pytest.fixture(scope="module")
def L():
    return ensure_built().lib()


@pytest.mark.parametrize("d", [64, 128])
def test_every_code_has_a_byte_of_its_own(d):
    at = int8.record_positions(d)
    assert sorted(at.ravel().tolist()) == list(range(32 * d))
    runs = at.reshape(2, 16, d // 8, 8)                    # eight dims of a token lie together, aligned
    assert (np.diff(runs, axis=-1) == 1).all() and (runs[..., 0] % 8 == 0).all()
    assert (at[0].reshape(16, -1, 64)[:, :, 0] % 64 == 0).all()


def test_new_scale_grows_by_two_at_least_or_stays():
    s = np.float32
    old = s(0.01)
    assert int8.new_scale(1.0, s(0)) == s(1.0) / s(127)
    assert int8.new_scale(1.27, old) == old or int8.new_scale(1.27, old) == s(0.02)
    assert int8.new_scale(1.26, old) == old
    assert int8.new_scale(1.30, old) == s(0.02)
    assert int8.new_scale(12.7, old) == s(12.7) / s(127)
    assert int8.new_scale(0.0, s(0)) == 0 and int8.new_scale(2.0 ** -94, s(0)) == 0
    assert np.isnan(int8.new_scale(np.inf, old)) and np.isnan(int8.new_scale(np.nan, old))
    assert np.isnan(int8.new_scale(1.0, s(np.nan)))


def test_rounding_of_kept_rows_stays_within_a_step():
    """A row written first and kept while a scale grows 15 times."""
    rng = np.random.default_rng(0)
    for growth in (1.001, 1.3, 2.0, 5.0):
        pool = np.zeros((1, 1, 32 * 64 + 16), np.uint8)
        x = rng.standard_normal((16, 1, 64)) * growth ** np.arange(16)[:, None, None]
        for t in range(16):
            int8.write_rows(x[t:t + 1], np.array([t]), pool, 0, 64)
            got = int8.dequant(pool, 64)[0][0, :, :t + 1].transpose(1, 0, 2)
            assert (np.abs(got - x[:t + 1]) <= int8.scales(pool)[0, 0, 0] * (1 + 2.0 ** -20)).all()
            assert (int8.codes(pool, 64)[0][0, 0, t + 1:] == 0).all()      # rows after the last: zeros


def test_a_write_of_a_whole_block_rounds_each_value_once():
    rng = np.random.default_rng(1)
    pool = rng.integers(0, 256, (3, 2, 32 * 128 + 16), dtype=np.uint8)
    x = rng.standard_normal((16, 2, 128))
    int8.write_rows(x, 16 + np.arange(16), pool, 1, 128)
    s = int8.scales(pool)[1, :, 1]
    got = int8.dequant(pool, 128)[1][1].transpose(1, 0, 2)
    assert (np.abs(got - x) <= s[None, :, None] * (0.5 + 2.0 ** -16)).all()
    assert np.allclose(s, np.abs(x).max((0, 2)) / 127, rtol=2.0 ** -23)


def test_norm_rope_has_its_invariants():
    """Rows of weight 1 have mean square 1 whatever their size and position."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 3, 64)) * 10.0 ** rng.integers(-2, 3, (5, 1, 1))
    for style in (oracle.ROPE_NEOX, oracle.ROPE_GPTJ, oracle.ROPE_NONE):
        y = int8.norm_rope(x, np.ones(64), 1e-12, np.arange(5) * 1000, 1e4, style)
        assert np.allclose((y * y).mean(-1), 1, rtol=1e-6)
    assert np.allclose(int8.norm_rope(x, None, 1.0, np.zeros(5), 1e4), x)


# ---- models of the kernels' arithmetic -------------------------------------------

def _f(x):
    return np.float32(x)


def _fma(a, b, c):
    """fp32 fma of arrays: the product is exact in long double, the sum rounded there to 64 bits first."""
    return (a.astype(np.longdouble) * np.longdouble(b) + np.asarray(c, np.longdouble)).astype(np.float32)


def test_the_corrected_product_is_the_quotient_by_127():
    """q = m fl(1/127), corrected once by its exact residual, for every mantissa
    and exponents from the least scale to the largest float."""
    mant = np.arange(1 << 23, dtype=np.uint32)
    inv = _f(1) / _f(127)
    for e in (34, 127, 253):
        m = ((np.uint32(e) << np.uint32(23)) | mant).view(np.float32)
        q = m * inv
        assert np.array_equal(_fma(_fma(q, -127.0, m), inv, q), m / _f(127))


def test_rotation_table_is_within_its_bound():
    """cos and sin of a fraction of a turn: the nearest quarter off exactly, the
    rest by Taylor series in fp32, within 2^-23 for fractions of every kind."""
    rng = np.random.default_rng(0)
    turn = np.concatenate([rng.integers(0, 2 ** 32, 1 << 20, dtype=np.uint64), np.arange(0, 2 ** 32, 2 ** 13, dtype=np.uint64),
                           (np.arange(9, dtype=np.uint64) * 2 ** 29 + np.arange(-3, 4)[:, None].astype(np.uint64)).ravel() & 0xFFFFFFFF])
    up = (turn + 0x20000000) & 0xFFFFFFFF
    rest = (up & 0x3FFFFFFF).astype(np.int64) - 0x20000000
    x = rest.astype(np.float32) * _f(2 * np.pi * 2.0 ** -32)
    x2 = x * x
    s = _fma(x2, _f(1 / 362880), _f(-1 / 5040))
    for k in (1 / 120, -1 / 6):
        s = _fma(x2, s.astype(np.longdouble), _f(k))
    s = _fma(x * x2, s.astype(np.longdouble), x)
    c = _fma(x2, _f(-1 / 3628800), _f(1 / 40320))
    for k in (-1 / 720, 1 / 24, -0.5, 1.0):
        c = _fma(x2, c.astype(np.longdouble), _f(k))
    quarter = (up >> 30).astype(int)
    sign = np.where(quarter >= 2, -1, 1)
    cos, sin = np.where(quarter & 1, -s, c) * sign, np.where(quarter & 1, c, s) * sign
    ang = turn.astype(np.float64) * (2 * np.pi / 2 ** 32)
    assert np.abs(cos - np.cos(ang)).max() <= 2.0 ** -23 and np.abs(sin - np.sin(ang)).max() <= 2.0 ** -23


def test_turns_of_far_positions():
    """The leading half of pos * F mod 2^64, taken from two 32-bit products."""
    rng = np.random.default_rng(1)
    for _ in range(2000):
        f, pos = int(rng.integers(0, 2 ** 63)) * 2 + int(rng.integers(0, 2)), int(rng.integers(0, 2 ** 31))
        lead = ((pos * (f & 0xFFFFFFFF) >> 32) + pos * (f >> 32)) & 0xFFFFFFFF
        assert lead == (pos * f % 2 ** 64) >> 32


def test_codes_are_the_low_bytes_of_one_fma():
    """fma(y, r, 1.5 * 2^23 + 128): its low byte is the code + 128, halves to even."""
    rng = np.random.default_rng(2)
    y = np.concatenate([rng.uniform(-127, 127, 20000), np.arange(-254, 255) / 2]).astype(np.float32)
    for r in (_f(1), _f(0.37), _f(1 / 3)):
        q = _fma(y, r, _f(12582912 + 128))
        assert np.array_equal((q.view(np.uint32) & 0xFF).astype(int) - 128, int8.round_codes(y, r))


P = ctypes.c_void_p


def _norm(L, int8_pool=False, **kw):
    a = dict(q=16, qpos=16, Tq=2, Hq=4, k=16, v=16, pos=16, slots=16, wq=16, wk=16, eps=1e-6, kc=16, vc=16, T=2, H=2,
             d=64, bs=16, nb=8, dt=1, theta=1e4, style=0)
    a.update(kw)
    head = [P(a["q"]), P(a["qpos"]), a["Tq"], a["Hq"], P(a["k"]), P(a["v"]), P(a["pos"]), P(a["slots"]), P(a["wq"]),
            P(a["wk"]), a["eps"], P(a["kc"])] + ([] if int8_pool else [P(a["vc"])])
    f = L.photon_qk_norm_rope_kv_cache_write_int8 if int8_pool else L.photon_qk_norm_rope_kv_cache_write
    return f(*head, a["T"], a["H"], a["d"], a["bs"], a["nb"], a["dt"], a["theta"], a["style"], None)


@pytest.mark.parametrize("pool", [False, True])
def test_norm_writes_refuse_before_any_launch(L, pool):
    f = lambda **kw: _norm(L, pool, **kw)
    for kw in (dict(T=-1), dict(Tq=-1), dict(H=0), dict(d=0), dict(nb=0), dict(dt=2), dict(style=9), dict(theta=-1.0),
               dict(theta=float("inf")), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(q=0), dict(qpos=0), dict(wq=0), dict(Hq=0), dict(k=0), dict(v=0), dict(pos=0), dict(slots=0), dict(wk=0),
               dict(kc=0), dict(q=24), dict(k=8), dict(v=40), dict(wk=4), dict(wq=8), dict(kc=8), dict(pos=2), dict(slots=4)):
        assert f(**kw) == -1, kw
    if not pool:
        assert f(vc=0) == -1 and f(vc=8) == -1
        assert f(d=512) == -2
    else:
        assert f(d=32) == -2 and f(d=256) == -2 and f(H=1025) == -2 and f(nb=2 ** 31) == -2
    assert f(bs=32) == -2 and f(d=96) == -2
    assert f(T=0, Tq=0, q=0, k=0) == 0
    assert f(T=0, Tq=0, style=2, theta=-1.0) == 0             # theta unused without rotation


def _write(L, **kw):
    a = dict(k=16, v=16, pos=16, slots=16, pool=16, T=2, H=2, d=64, bs=16, nb=8, dt=1, theta=1e4, style=0)
    a.update(kw)
    return L.photon_kv_cache_write_int8(P(a["k"]), P(a["v"]), P(a["pos"]), P(a["slots"]), P(a["pool"]), a["T"], a["H"], a["d"],
                                        a["bs"], a["nb"], a["dt"], a["theta"], a["style"], None)


def _read(L, **kw):
    a = dict(pool=16, slots=16, k=16, v=16, T=2, H=2, d=64, bs=16, nb=8, dt=1)
    a.update(kw)
    return L.photon_kv_cache_read_int8(P(a["pool"]), P(a["slots"]), P(a["k"]), P(a["v"]), a["T"], a["H"], a["d"], a["bs"], a["nb"],
                                       a["dt"], None)


def _decode(L, **kw):
    a = dict(q=16, pool=16, bt=16, cl=16, scale=0.125, out=16, B=2, Hq=8, Hkv=2, d=64, bs=16, nb=100, W=4, mc=64, part=512, odt=0,
             ws=0, wsb=0)
    a.update(kw)
    return L.photon_paged_attention_decode_int8(P(a["q"]), P(a["pool"]), P(a["bt"]), P(a["cl"]), a["scale"], P(a["out"]), a["B"],
                                                a["Hq"], a["Hkv"], a["d"], a["bs"], a["nb"], a["W"], a["mc"], a["part"], a["odt"],
                                                P(a["ws"]), a["wsb"], None)


def test_int8_calls_refuse_before_any_launch(L):
    for f in (_write, _read):
        for kw in (dict(T=-1), dict(H=0), dict(d=-4), dict(nb=0), dict(dt=7), dict(k=0), dict(v=0), dict(slots=0), dict(pool=0),
                   dict(k=8), dict(v=4), dict(pool=8), dict(slots=4)):
            assert f(L, **kw) == -1, (f, kw)
        for kw in (dict(d=32), dict(d=256), dict(bs=8), dict(H=2000), dict(nb=2 ** 31)):
            assert f(L, **kw) == -2, (f, kw)
        assert f(L, T=0, k=0, v=0) == 0
    assert _write(L, theta=0.0) == -1 and _write(L, pos=0) == -1 and _write(L, style=3) == -1
    for kw in (dict(q=0), dict(q=8), dict(pool=24), dict(out=20), dict(bt=0), dict(cl=0), dict(Hq=6, Hkv=4), dict(part=100), dict(W=3),
               dict(scale=float("nan")), dict(odt=5), dict(B=-1)):
        assert _decode(L, **kw) == -1, kw
    for kw in (dict(d=32), dict(d=256), dict(bs=8), dict(Hq=32), dict(Hq=2048, Hkv=2048), dict(nb=2 ** 31), dict(mc=2 ** 31 - 16, W=2 ** 27, part=2 ** 30, ws=256, wsb=1 << 60)):
        assert _decode(L, **kw) == -2, kw
    assert _decode(L, mc=1024, W=64) == -3                   # split needed, no workspace
    assert _decode(L, B=0) == 0
    assert L.photon_kv_cache_int8_record_bytes(64) == 2064 and L.photon_kv_cache_int8_record_bytes(128) == 4112
    assert L.photon_kv_cache_int8_record_bytes(32) == 0 and L.photon_kv_cache_int8_record_bytes(-1) == 0
