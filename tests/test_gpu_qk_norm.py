"""q/k RMS norms, rotation and cache write in one launch, on the GPU against the
fp64 definition (oracle/int8.py norm_rope)."""
import numpy as np
import pytest

import oracle
import synth
from oracle import int8
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu

STYLES = {"neox": oracle.ROPE_NEOX, "gptj": oracle.ROPE_GPTJ, "none": oracle.ROPE_NONE}
CACHE = -5.0


def _torch():
    import torch
    return torch


def _dev(a):
    return _torch().from_numpy(np.ascontiguousarray(a)).cuda()


def _storage(x, dtype):
    """A float array as storage: float32, or bf16 bits (uint16) and its tensor."""
    torch = _torch()
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32))
    t = t if dtype == "f32" else t.bfloat16()
    return synth.to_storage_numpy(t), t.cuda()


def _allowed(y, style, dtype):
    """Half a step of the type and, before it, 2^-19 of the pair's length:
      mean square: 8 products and sums per lane, at most 5 more sums, eps: 14
        roundings of 2^-24, halved by the root; rsqrt 2 ulp (2^-22), two products:
        (7 + 4 + 2) 2^-24 < 2^-20
      rotation: cos and sin within 2^-23 + 2^-29, two products and a sum:
        at most 2^-22 (|a| + |b|) <= 2^-21.5 of the length
    A value below the type's normal numbers is off by at most a step of 2^-126."""
    return (np.abs(y) * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24)
            + int8.pair_length(y, STYLES[style]) * 2.0 ** -19 + 2.0 ** -126)


def _run(T, H, Tq, Hq, d, dtype, style, rng, pos=None, qpos=None, kscale=1.0, theta=1e6, eps=1e-6, skip=True):
    """One call on random inputs; checks every element of q and of both pools."""
    torch = _torch()
    pk = ensure_built()
    nb = T // 16 + 5
    k, kt = _storage(rng.standard_normal((T, H, d)) * kscale, dtype)
    v, vt = _storage(rng.standard_normal((T, H, d)), dtype)
    q, qt = _storage(rng.standard_normal((Tq, Hq, d)) * kscale, dtype)
    wk, wkt = _storage(1 + 0.3 * rng.standard_normal(d), dtype)
    wq, wqt = _storage(1 + 0.3 * rng.standard_normal(d), dtype)
    pos = rng.integers(0, 2 ** 20, T).astype(np.int32) if pos is None else pos
    qpos = rng.integers(0, 2 ** 20, Tq).astype(np.int32) if qpos is None else qpos
    slots = rng.permutation(nb * 16)[:T].astype(np.int64)
    gpu_slots = slots.copy()
    if skip and T > 4:
        gpu_slots[3::7] = -1
        gpu_slots[3::14] = nb * 16 + 2
    live = (gpu_slots >= 0) & (gpu_slots < nb * 16)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    kc, vc = (torch.full((nb, H, 16, d), CACHE, dtype=dt, device="cuda") for _ in range(2))
    pk.photon_device_errors()
    pk.photon_qk_norm_rope_kv_cache_write(qt, _dev(qpos), kt, vt, _dev(pos), _dev(gpu_slots), wqt, wkt, eps, kc, vc,
                                          theta, style)
    torch.cuda.synchronize()
    assert pk.photon_device_errors() == (pk.DEVERR_SLOT_RANGE if (gpu_slots >= nb * 16).any() else 0)
    yq = int8.norm_rope(q, wq, eps, qpos, theta, STYLES[style])
    yk = int8.norm_rope(k, wk, eps, pos, theta, STYLES[style])
    assert (np.abs(qt.double().cpu().numpy() - yq) <= _allowed(yq, style, dtype)).all()
    want_v = torch.full_like(vc, CACHE)
    b, o = slots[live] // 16, slots[live] % 16
    want_v[_dev(b), :, _dev(o)] = vt[_dev(np.nonzero(live)[0])]
    assert torch.equal(vc, want_v)
    got = kc.double().cpu().numpy()
    assert (np.abs(got[b, :, o] - yk[live]) <= _allowed(yk[live], style, dtype)).all()
    got[b, :, o] = CACHE
    assert (got == CACHE).all()                          # slots of no token


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("style", ["neox", "gptj", "none"])
@pytest.mark.parametrize("T,H,Tq,Hq", [(1, 1, 1, 1), (5, 3, 7, 6), (23, 8, 23, 16)])
def test_rows_match_the_definition(T, H, Tq, Hq, style, dtype, d):
    _run(T, H, Tq, Hq, d, dtype, style, np.random.default_rng(T + d))


@pytest.mark.parametrize("T,H,Tq,Hq,d", [(700, 1, 31, 5, 64), (1300, 2, 0, 2, 128), (0, 3, 1259, 2, 64), (2501, 1, 2437, 1, 32),
                                         (310, 2, 640, 3, 256)])
def test_tiles_of_several_tokens(T, H, Tq, Hq, d):
    """More tokens than CTAs of one token: tiles with a ragged end; queries or
    keys alone."""
    _run(T, H, Tq, Hq, d, "bf16", "neox", np.random.default_rng(T + Tq))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("style", ["neox", "gptj"])
def test_far_positions(style, dtype):
    pos = np.array([0, 1, 2, 2 ** 30, 2 ** 31 - 1, 123456789], np.int32)
    for theta in (1e4, 1e6, 0.5):
        _run(6, 2, 6, 3, 128, dtype, style, np.random.default_rng(3), pos=pos, qpos=pos[::-1].copy(), theta=theta,
             skip=False)


@pytest.mark.parametrize("kscale", [2.0 ** -70, 2.0 ** -10, 2.0 ** 55])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_magnitudes(kscale, dtype):
    """Rows far below eps, near it, and as large as squares fit fp32."""
    _run(9, 2, 9, 4, 64, dtype, "neox", np.random.default_rng(4), kscale=kscale)


def test_zero_rows_and_non_finite_rows():
    """A row of zeros stays zero; an infinity or a NaN makes its row NaN (or zero
    and NaN, infinity over infinity) and no other."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(5)
    T, H, d = 6, 2, 64
    x = rng.standard_normal((T, H, d)).astype(np.float32)
    x[0], x[2, 1, 7], x[3, 0, 40] = 0, np.inf, np.nan
    w = torch.ones(d, device="cuda")
    kc, vc = (torch.zeros(1, H, 16, d, device="cuda") for _ in range(2))
    q = _dev(x)
    pos = _dev(np.zeros(T, np.int32))
    pk.photon_qk_norm_rope_kv_cache_write(q, pos, _dev(x), _dev(x), pos, _dev(np.arange(T)), w, w, 1e-6, kc, vc, 1e4)
    for y in (q, kc[0, :, :T].transpose(0, 1)):
        bad = torch.isnan(y).any(-1).cpu().numpy()
        want = np.zeros((T, H), bool)
        want[2, 1] = want[3, 0] = True
        assert np.array_equal(bad, want)
        assert (y[0] == 0).all()
    assert torch.equal(vc[0, :, :T].transpose(0, 1).nan_to_num(), _dev(x).nan_to_num())


def test_on_another_stream_and_captured():
    """The same bits on a side stream and replayed from a graph with new inputs."""
    torch = _torch()
    pk = ensure_built()
    gen = torch.Generator(device="cuda").manual_seed(1)
    T, H, Hq, d = 33, 4, 8, 128
    mk = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
    k, v, q0, wq, wk = mk(T, H, d), mk(T, H, d), mk(T, Hq, d), mk(d), mk(d)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 11
    slots = torch.randperm(64, generator=gen, device="cuda")[:T]
    call = lambda q, kc, vc, **kw: pk.photon_qk_norm_rope_kv_cache_write(q, pos, k, v, pos, slots, wq, wk, 1e-5, kc, vc, 1e4, **kw)
    pools = lambda: [torch.zeros(4, H, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q1, p1 = q0.clone(), pools()
    call(q1, *p1)
    q2, p2 = q0.clone(), pools()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(q2, *p2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(q1, q2) and all(torch.equal(a, b) for a, b in zip(p1, p2))
    q3, p3 = q0.clone(), pools()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(q3, *p3)
    q3.copy_(q0)
    g.replay()
    assert torch.equal(q1, q3) and all(torch.equal(a, b) for a, b in zip(p1, p3))
    k.mul_(-1)
    q3.copy_(q0)
    g.replay()
    assert torch.equal(p3[0], -p1[0]) and torch.equal(q1, q3)


def test_equals_norm_then_rotation_then_write():
    """What the call replaces: norms in fp32, rounded once less, then the rotating
    write.  Both are within a step of the type of each other."""
    torch = _torch()
    pk = ensure_built()
    gen = torch.Generator(device="cuda").manual_seed(2)
    T, H, Hq, d = 40, 8, 16, 128
    k, v, q = (torch.randn(T, n, d, generator=gen, device="cuda") for n in (H, H, Hq))
    w = 1 + 0.1 * torch.randn(d, generator=gen, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 1000
    slots = torch.arange(T, device="cuda") + 16
    norm = lambda x: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
    a, b = ([torch.zeros(4, H, 16, d, device="cuda") for _ in range(2)] for _ in range(2))
    qa, qb = norm(q).contiguous(), q.clone()
    pk.photon_rope_q_kv_cache_write(qa, pos, norm(k).contiguous(), v, pos, slots, *a, 1e6)
    pk.photon_qk_norm_rope_kv_cache_write(qb, pos, k, v, pos, slots, w, w, 1e-6, *b, 1e6)
    assert torch.equal(a[1], b[1])
    # each is within 2^-19 of a pair's length; normalised rows of weight 1.5 at most have lengths below 1.5 sqrt(128)
    for x, y in ((qa, qb), (a[0], b[0])):
        assert (x - y).abs().max().item() <= 2 * 1.5 * 128 ** 0.5 * 2.0 ** -19


def test_pools_past_32_bits():
    """Slots at the end of pools of more than 2^31 elements."""
    torch = _torch()
    pk = ensure_built()
    gen = torch.Generator(device="cuda").manual_seed(6)
    T, H, d, nb = 37, 2, 128, 600000
    k, v = (torch.randn(T, H, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    out = []
    for blocks in (nb, 3):
        kc, vc = (torch.empty(blocks, H, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        slots = (blocks - 3) * 16 + torch.arange(T, device="cuda")
        pk.photon_qk_norm_rope_kv_cache_write(None, None, k, v, pos, slots, None, w, 1e-6, kc, vc, 1e4)
        out.append([c[-3:].transpose(1, 2).reshape(48, H, d)[:T].clone() for c in (kc, vc)])
    assert all(torch.equal(a, b) for a, b in zip(*out)) and torch.equal(out[0][1], v)
    assert pk.photon_device_errors() == 0


def test_refusals():
    torch = _torch()
    pk = ensure_built()
    T, H, d = 4, 2, 64
    f = dict(dtype=torch.bfloat16, device="cuda")
    q, k, v, w = torch.zeros(T, 4, d, **f), torch.zeros(T, H, d, **f), torch.zeros(T, H, d, **f), torch.zeros(d, **f)
    pos, slots = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.arange(T, device="cuda")
    kc, vc = torch.zeros(2, H, 16, d, **f), torch.zeros(2, H, 16, d, **f)
    good = dict(q=q, q_positions=pos, k=k, v=v, positions=pos, slot_mapping=slots, q_weight=w, k_weight=w, eps=1e-6,
                k_cache=kc, v_cache=vc, rope_theta=1e4)
    call = lambda **kw: pk.photon_qk_norm_rope_kv_cache_write(**{**good, **kw})
    call()
    call(q=None, q_positions=None, q_weight=None)
    for kw in (dict(q=q.float()), dict(k_weight=w.float()), dict(v=v[:2]), dict(positions=pos.long()),
               dict(slot_mapping=slots.int()), dict(k=k.transpose(0, 1)), dict(v_cache=vc[:1]), dict(k_cache=kc[0]),
               dict(q_weight=w[:32].contiguous()), dict(q=q[..., :32].contiguous()), dict(positions=pos.cpu()),
               dict(k=k.cpu()), dict(k=k.double(), v=v.double(), q=q.double())):
        with pytest.raises((TypeError, ValueError, pk.PhotonError)):
            call(**kw)
    for kw in (dict(eps=0.0), dict(eps=float("nan")), dict(eps=-1e-6), dict(rope_theta=-1.0), dict(rope_style=7)):
        with pytest.raises(pk.PhotonError):
            call(**kw)
    assert pk.photon_device_errors() == 0
