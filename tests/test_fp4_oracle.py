"""CPU checks of the 4-bit KV cache and the device step metadata: the oracle's
definitions pinned to something other than themselves, and every refusal that
the calls make on the host before a launch."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

import oracle
import synth
from oracle import fp4
from tests.helpers import ensure_built


def test_e2m1_values():
    assert fp4.VALUES[:8].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert (fp4.VALUES[8:] == -fp4.VALUES[:8]).all()


def test_encode_is_the_nearest_code_with_ties_to_even():
    """Against exact rationals: midpoints, a hair beside them, random values."""
    rng = np.random.default_rng(0)
    scales = [float(np.float32(m) * 2.0 ** -9) for m in (128, 129, 200, 255)]
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    for s in scales:
        ys = [m * s for m in mids] + [m * s * (1 + d) for m in mids for d in (2.0 ** -20, -2.0 ** -20)]
        ys += list(rng.standard_normal(50).astype(np.float32).astype(float) * 3 * s) + [100 * s, 0.0]
        for y in ys:
            q = abs(Fraction(y)) / Fraction(s)
            d = [abs(q - Fraction(float(v))) for v in fp4.VALUES[:8]]
            best = [c for c in range(8) if d[c] == min(d)]
            want = best[0] if len(best) == 1 else [c for c in best if c % 2 == 0][0]
            got = int(fp4.encode(np.array([y]), np.array([s]))[0])
            assert got & 7 == want and (got >> 3) == (y < 0), (y, s)


@pytest.mark.parametrize("d", [64, 128])
def test_record_positions_are_a_bijection_and_private_to_a_token(d):
    byte, nib, sb = fp4.record_positions(d)
    owners = {}
    for w in range(2):
        for r in range(16):
            mine = set(byte[w, r]) | set(sb[w, r]) | set(sb[w, r] + 1)
            assert len(mine) == d // 2 + 2 * (d // 64)
            for b in mine:
                assert owners.setdefault(int(b), (w, r)) == (w, r)
    assert sorted(owners) == list(range(17 * d))
    assert len({(int(b), int(n)) for w in range(2) for r in range(16) for b, n in zip(byte[w, r], nib)}) == 32 * d


@pytest.mark.parametrize("d", [64, 128])
def test_write_then_dequant_is_within_half_a_step(d):
    """|value - y| <= scale (the widest gap, 4 to 6, is 2 scales; the largest
    magnitude is 6 scales up to the scale's own rounding, 2^-8 of 6 scales)."""
    rng = np.random.default_rng(d)
    T, H = 9, 2
    k, v = (rng.standard_normal((T, H, d)).astype(np.float32) for _ in range(2))
    pool = np.zeros((3, H, 17 * d), np.uint8)
    slots = rng.permutation(48)[:T].astype(np.int64)
    pos = np.arange(T, dtype=np.int32)
    fp4.write(k, v, pos, slots, pool, 1e4)
    kd, vd = fp4.dequant(pool, d)
    want = oracle.rope_rows(k, pos, 1e4)
    for t in range(T):
        b, r = divmod(int(slots[t]), 16)
        for got, y in ((kd[b, :, r], want[t]), (vd[b, :, r], v[t])):
            s = np.repeat(np.abs(y.reshape(H, -1, 64)).max(-1) / 6, 64, -1).reshape(H, d)
            assert (np.abs(got - y) <= s * (1 + 6 * 2.0 ** -8)).all()


def test_quantise_special_groups():
    y = np.zeros((4, 64), np.float32)
    y[1, 3] = np.inf
    y[2, 5] = np.nan
    y[3] = 2.0 ** -130                     # a subnormal bf16 scale
    codes, bits = fp4.quantise(y)
    assert bits[0, 0] == 0 and not codes[0].any()
    assert bits[1, 0] == bits[2, 0] == 0x7FFF
    sc = oracle.bf16_to_f64(bits[3])[0]
    # a subnormal scale is off by up to half of 2^-133, the largest magnitude (6 scales) by six times
    # that; the codes add one scale (half of the widest gap)
    assert 0 < sc < 2.0 ** -126
    assert np.abs(fp4.VALUES[codes[3]] * sc - 2.0 ** -130).max() <= sc + 6 * 2.0 ** -134


def test_step_metadata_oracle_equals_the_host_builder():
    """Without releases: the same lists, tables and pool as the host call."""
    pk = ensure_built()
    rng = np.random.default_rng(3)
    nb, W, B = 200, 12, 9
    pool = pk.BlockPool(nb, seed=5)
    order = pool.alloc(nb)          # the order in which this pool hands out
    pool = pk.BlockPool(nb, seed=5)
    bt = np.full((B, W), -1, np.int32)
    nc = np.zeros(B, np.int32)
    stack = [int(x) for x in order[::-1]]
    for step in range(4):
        nn = rng.integers(0, 40, B).astype(np.int32)
        tab, st, seq, pos, slots, ctx, status = fp4.step_metadata(nc, nn, bt, stack, int(nn.sum()), nb)
        got = pk.photon_build_step_metadata(nc, nn, bt, pool)
        assert status == 0 and np.array_equal(tab, bt) and len(st) == pool.num_free()
        assert got["token_seq"].tolist() == seq and got["positions"].tolist() == pos
        assert got["slot_mapping"].tolist() == slots and np.array_equal(got["context_lens"], ctx)
        nc, stack = ctx.astype(np.int32), st


# ---- refusals on the host ---------------------------------------------------------

P = ctypes.c_void_p


def _w(L, **kw):
    a = dict(k=16, v=16, pos=16, sm=16, kv=16, T=4, H=2, d=64, bs=16, nb=8, dt=1, theta=1e4, style=0)
    a.update(kw)
    return L.photon_kv_cache_write_fp4(P(a["k"]), P(a["v"]), P(a["pos"]), P(a["sm"]), P(a["kv"]), a["T"], a["H"],
                                       a["d"], a["bs"], a["nb"], a["dt"], a["theta"], a["style"], None)


def _r(L, **kw):
    a = dict(k=16, v=16, sm=16, kv=16, T=4, H=2, d=64, bs=16, nb=8, dt=1)
    a.update(kw)
    return L.photon_kv_cache_read_fp4(P(a["kv"]), P(a["sm"]), P(a["k"]), P(a["v"]), a["T"], a["H"], a["d"], a["bs"],
                                      a["nb"], a["dt"], None)


def _d(L, **kw):
    a = dict(q=16, kv=16, bt=16, cl=16, scale=0.125, out=16, B=2, Hq=8, Hkv=2, d=64, bs=16, nb=100, W=4, mc=64,
             part=512, odt=0, ws=0, wsb=0)
    a.update(kw)
    return L.photon_paged_attention_decode_fp4(P(a["q"]), P(a["kv"]), P(a["bt"]), P(a["cl"]), a["scale"], P(a["out"]),
                                               a["B"], a["Hq"], a["Hkv"], a["d"], a["bs"], a["nb"], a["W"], a["mc"],
                                               a["part"], a["odt"], P(a["ws"]), a["wsb"], None)


def _m(L, **kw):
    a = dict(nc=1 << 20, nn=2 << 20, B=4, bs=16, bt=3 << 20, W=8, fb=4 << 20, nb=64, nf=5 << 20, nfo=5 << 20, M=16,
             ts=6 << 20, pos=7 << 20, sm=8 << 20, cl=9 << 20, tot=10 << 20)
    a.update(kw)
    return L.photon_build_step_metadata_device(P(a["nc"]), P(a["nn"]), a["B"], a["bs"], P(a["bt"]), a["W"],
                                               P(a["fb"]), a["nb"], P(a["nf"]), P(a["nfo"]), a["M"], P(a["ts"]),
                                               P(a["pos"]), P(a["sm"]), P(a["cl"]), P(a["tot"]), None)


@pytest.mark.parametrize("call,bad", [
    (_w, dict(k=0)), (_w, dict(v=0)), (_w, dict(pos=0)), (_w, dict(sm=0)), (_w, dict(kv=0)), (_w, dict(k=8)),
    (_w, dict(kv=24)), (_w, dict(sm=4)), (_w, dict(pos=2)), (_w, dict(T=-1)), (_w, dict(H=0)), (_w, dict(nb=0)),
    (_w, dict(dt=3)), (_w, dict(style=5)), (_w, dict(theta=0.0)), (_w, dict(theta=float("inf"))),
    (_w, dict(nb=2 ** 62)),
    (_r, dict(k=0)), (_r, dict(v=8)), (_r, dict(kv=0)), (_r, dict(sm=12)), (_r, dict(T=-1)), (_r, dict(dt=2)),
    (_r, dict(H=-1)), (_r, dict(nb=0)),
    (_d, dict(q=0)), (_d, dict(kv=0)), (_d, dict(bt=0)), (_d, dict(cl=0)), (_d, dict(out=0)), (_d, dict(out=8)),
    (_d, dict(scale=float("nan"))), (_d, dict(Hq=7)), (_d, dict(part=24)), (_d, dict(W=3)), (_d, dict(odt=4)),
    (_d, dict(B=-1)),
    (_m, dict(nc=0)), (_m, dict(nn=0)), (_m, dict(bt=0)), (_m, dict(fb=0)), (_m, dict(nf=0)), (_m, dict(nfo=0)),
    (_m, dict(ts=0)), (_m, dict(pos=0)), (_m, dict(sm=0)), (_m, dict(cl=0)), (_m, dict(tot=0)), (_m, dict(B=-1)),
    (_m, dict(M=-1)), (_m, dict(W=0)), (_m, dict(nb=0)), (_m, dict(bs=0)), (_m, dict(sm=(8 << 20) + 4)),
    (_m, dict(cl=1 << 20)), (_m, dict(cl=(2 << 20) + 12)), (_m, dict(nc=(1 << 20) + 1)),
])
def test_invalid_arguments_are_refused(call, bad):
    assert call(ensure_built().lib(), **bad) == -1


@pytest.mark.parametrize("call,bad", [
    (_w, dict(d=32)), (_w, dict(d=256)), (_w, dict(d=96)), (_w, dict(bs=32)), (_w, dict(nb=2 ** 31)), (_w, dict(H=1025)), (_d, dict(Hkv=1025, Hq=1025)), (_r, dict(nb=2 ** 31)), (_r, dict(d=256)), (_r, dict(bs=8)),
    (_d, dict(d=32)), (_d, dict(d=256)), (_d, dict(Hq=6)), (_d, dict(Hq=32)), (_d, dict(bs=8)), (_d, dict(mc=2 ** 31 - 16, W=2 ** 27, part=2 ** 30, ws=256, wsb=2 ** 40)),
    (_m, dict(bs=32)), (_m, dict(B=16385)), (_m, dict(nb=2 ** 31)), (_m, dict(B=16384, W=2 ** 17)),
])
def test_unsupported_shapes_are_refused(call, bad):
    assert call(ensure_built().lib(), **bad) == -2


def test_small_workspace_is_refused():
    L = ensure_built().lib()
    need = L.photon_paged_attention_workspace_size(2, 8, 64, 64, 16)
    assert _d(L, part=16) == -3 and _d(L, part=16, ws=256, wsb=need - 1) == -3


def test_empty_calls_do_nothing():
    L = ensure_built().lib()
    assert _w(L, T=0, k=0) == 0 and _r(L, T=0, k=0) == 0 and _d(L, B=0, q=0) == 0
    assert L.photon_kv_cache_fp4_record_bytes(64) == 1088 and L.photon_kv_cache_fp4_record_bytes(128) == 2176
    assert L.photon_kv_cache_fp4_record_bytes(32) == 0


def test_binding_refuses_wrong_tensors():
    """Tensors of the host, of other types or shapes raise before the library is called."""
    import torch
    pk = ensure_built()
    kv = torch.zeros(4, 2, 17 * 64, dtype=torch.uint8)
    x = torch.zeros(3, 2, 64)
    i32, i64 = torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        pk.photon_kv_cache_write_fp4(x, x, i32, i64, kv, 1e4)
    with pytest.raises(ValueError):
        pk.photon_kv_cache_read_fp4(kv, i64, x, x)
    with pytest.raises(ValueError):
        pk.photon_paged_attention_decode_fp4(x.bfloat16(), kv, i32.view(3, 1), i32, 1.0, x, 16)
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        pk.photon_build_step_metadata_device(i32, i32, i32.view(3, 1), i32, one, i32, i32, i64, i32, one)
