"""Query rows of the normalising 8-bit write around the count from which they get
a launch of their own, every row against the definition in 64 bits."""
import numpy as np
import pytest

from oracle import int8
from tests.helpers import ensure_built
from tests.test_gpu_launch_shapes import launches

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _definition(x, w, eps, pos, theta):
    """Norm and rotation by halves of [T, H, d] in 64 bits, and the length of each value's pair."""
    torch = _torch()
    x = x.double()
    y = x * w.double() / (x.square().mean(-1, keepdim=True) + float(np.float32(eps))).sqrt()
    half = y.shape[-1] // 2
    freq = theta ** (-torch.arange(half, dtype=torch.float64, device=x.device) / half)
    ang = pos.double()[:, None, None] * freq
    a, b = y[..., :half], y[..., half:]
    n = torch.hypot(a, b)
    return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1), torch.cat([n, n], -1)


@pytest.mark.parametrize("d,Hq,rows", [(64, 32, 524288), (128, 16, 131072)])
@pytest.mark.parametrize("less", [1, 0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_queries_around_the_launch_of_their_own(d, Hq, rows, less, dtype):
    """Allowed: half a step of the type and 2^-19 of the pair's length, as the write states."""
    torch = _torch()
    pk = ensure_built()
    gen = torch.Generator(device="cuda").manual_seed(rows + less)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    Tq, T, H, nb, theta, eps = rows // Hq - less, 35, 2, 5, 1e6, 1e-6
    q = torch.randn(Tq, Hq, d, generator=gen, device="cuda").to(dt)
    k, v = (torch.randn(T, H, d, generator=gen, device="cuda").to(dt) for _ in range(2))
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dt) for _ in range(2))
    qpos = torch.randint(0, 2 ** 20, (Tq,), generator=gen, device="cuda").int()
    pos = torch.arange(T, device="cuda").int() + 77
    slots = torch.arange(T, device="cuda") + 3
    start = torch.zeros(nb, H, 32 * d + 16, dtype=torch.uint8, device="cuda")
    call = lambda q, pool, **kw: pk.photon_qk_norm_rope_kv_cache_write_int8(q, qpos, k, v, pos, slots, wq, wk, eps, pool, theta, **kw)
    names = [n[0].split("<")[0] for n in launches(lambda st: call(q, start, stream=st))]
    assert names == ([] if less else ["qk_norm_rope_write_kernel"]) + ["kv_cache_write_int8_kernel"]
    mine, pool = q.clone(), start.clone()
    call(mine, pool)
    step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for t in range(0, Tq, 2048):
        want, length = _definition(q[t:t + 2048], wq, eps, qpos[t:t + 2048], theta)
        assert ((mine[t:t + 2048].double() - want).abs() <= want.abs() * step + length * 2.0 ** -19).all(), t
    # the keys beside them: half a code, and what norm and rotation may be off by
    want, length = _definition(k, wk, eps, pos, theta)
    sc = torch.from_numpy(int8.scales(pool.cpu().numpy()).copy()).cuda()[slots // 16].double()
    kb, vb = (torch.empty(T, H, d, device="cuda") for _ in range(2))
    pk.photon_kv_cache_read_int8(pool, slots, kb, vb)
    half = 0.5 * (1 + 2.0 ** -15)       # codes up to 127 times 2^-24 of fl(1 / s) and of the product read back
    assert ((kb.double() - want).abs() <= half * sc[..., :1] + length * 2.0 ** -19).all()
    assert ((vb.double() - v.double()).abs() <= half * sc[..., 1:]).all()
    assert pk.photon_device_errors() == 0
