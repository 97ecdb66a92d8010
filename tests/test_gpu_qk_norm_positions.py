"""q/k norms at negative positions: padding rows of the step metadata have -1, and
their queries are rotated like any other row (their keys have slot -1)."""
import numpy as np
import pytest

from tests.helpers import ensure_built
from tests.test_gpu_qk_norm import _run, _torch

pytestmark = pytest.mark.gpu

NEGATIVE = np.array([-1, 0, -2, -2 ** 31, 2 ** 31 - 1, -1000003, 5], np.int32)


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("style", ["neox", "gptj"])
def test_negative_positions(style, dtype, d):
    n = len(NEGATIVE)
    _run(n, 2, n, 3, d, dtype, style, np.random.default_rng(d), pos=NEGATIVE, qpos=NEGATIVE[::-1].copy(), theta=1e4, skip=False)


@pytest.mark.parametrize("d", [64, 128])
def test_padding_rows_agree_with_the_bf16_write(d):
    """The 8-bit write's queries are those of the bf16 one, bit for bit, padding rows too."""
    torch = _torch()
    pk = ensure_built()
    gen = torch.Generator(device="cuda").manual_seed(d)
    T, H, Hq = 9, 2, 6
    mk = lambda h: torch.randn(T, h, d, generator=gen, device="cuda").bfloat16()
    q, k, v = mk(Hq), mk(H), mk(H)
    w = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).bfloat16()
    pos = torch.tensor([3, 4, 5, 6, -1, -1, -1, -1, -1], dtype=torch.int32, device="cuda")
    slots = torch.tensor([3, 4, 5, 6, -1, -1, -1, -1, -1], device="cuda")
    a, b = q.clone(), q.clone()
    pool = torch.zeros(1, H, 32 * d + 16, dtype=torch.uint8, device="cuda")
    kc, vc = (torch.zeros(1, H, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pk.photon_qk_norm_rope_kv_cache_write(a, pos, k, v, pos, slots, w, w, 1e-6, kc, vc, 1e4)
    pk.photon_qk_norm_rope_kv_cache_write_int8(b, pos, k, v, pos, slots, w, w, 1e-6, pool, 1e4)
    assert torch.equal(a, b)
    # and those of norm, then rotation: both within 2^-19 of a pair's length and half a bf16 step (2^-8)
    norm = q.double() * torch.rsqrt(q.double().square().mean(-1, keepdim=True) + 1e-6) * w.double()
    c = norm.float()
    pk.photon_rope_q_kv_cache_write(c, pos, k.float(), v.float(), pos, torch.full_like(slots, -1), kc.float(), vc.float(), 1e4)
    length = torch.hypot(c[..., :d // 2], c[..., d // 2:]).repeat(1, 1, 2)
    assert ((a.double() - c.double()).abs() <= c.double().abs() * 2.0 ** -8 + length * 2.0 ** -18).all()
    assert pk.photon_device_errors() == 0
