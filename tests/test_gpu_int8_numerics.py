"""Decode over the 8-bit cache: what its outputs keep of the 32-bit sums, and
inputs at the ends of the documented range."""
import numpy as np
import pytest

import oracle
from oracle import int8
from tests.helpers import bf16_spacing, ensure_built
from tests.test_gpu_int8 import DECLARED, _decode, _dev, _random_pool, _storage, _tables, _tolerance, _torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("declared", DECLARED)
@pytest.mark.parametrize("ctx,part,H,G,d", [
    ([16], 512, 8, 4, 64), ([1024], 32, 8, 4, 64), ([700, 33, 0, 5, 1500], 128, 4, 2, 128), ([3000, 200, 2500], 64, 2, 8, 64),
    ([200] * 40 + [1, 0], 64, 8, 1, 128), ([900] * 24, 512, 8, 4, 64), ([9000, 20000], 256, 4, 8, 128)])
def test_a_bf16_output_is_the_32_bit_one_rounded(ctx, part, H, G, d, declared):
    """The type of the output decides its last rounding and nothing before it:
    bit for bit the fp32 call's values rounded to bf16."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(sum(ctx) + d)
    nb = sum(-(-c // 16) for c in ctx) + 2
    bank = _random_pool(rng, min(nb, 64), H, d)
    pool = _dev(bank)[_dev(rng.integers(0, len(bank), nb))].contiguous()
    bt = _tables(rng, ctx, nb)
    _, qt = _storage(rng.standard_normal((len(ctx), H * G, d)), "bf16")
    fine = _decode(pk, qt, pool, bt, ctx, d ** -0.5, torch.float32, part, max_ctx=declared)
    coarse = _decode(pk, qt, pool, bt, ctx, d ** -0.5, torch.bfloat16, part, max_ctx=declared)
    assert torch.equal(coarse, fine.bfloat16())


@pytest.mark.parametrize("declared", DECLARED)
@pytest.mark.parametrize("d", [64, 128])
def test_bf16_outputs_are_off_by_half_a_step_of_their_own(d, declared):
    """With a softmax scale of zero every weight is the same, so its rounding moves
    all of a row alike.  Allowed: half the distance of bf16 numbers at the value, and
    what an fp32 output may be off by (weights within 2^-22)."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(d)
    H, G, ctx = 4, 4, [16, 48, 7, 640, 1]
    nb = sum(-(-c // 16) for c in ctx) + 2
    pool = _random_pool(rng, nb, H, d)
    bt = _tables(rng, ctx, nb)
    q, qt = _storage(rng.standard_normal((len(ctx), H * G, d)), "bf16")
    got = _decode(pk, qt, _dev(pool), bt, ctx, 0.0, torch.bfloat16, 64, max_ctx=declared).double().cpu().numpy()
    ref = int8.paged_attention(q, pool, bt, ctx, 0.0)
    kd, vd = int8.dequant(pool, d)
    fp32 = _tolerance(oracle.to_f64(q), kd, vd, ctx, 0.0, False, ref)
    assert (np.abs(got - ref) <= 0.5 * bf16_spacing(ref) + fp32).all()


def _set_k_scales(pool, factor):
    sc = int8.scales(pool).copy()
    sc[..., 0] = (sc[..., 0] / sc[..., 0].max() * factor).astype(np.float32)
    pool[:, :, -16:-8] = sc.view(np.uint8)


@pytest.mark.parametrize("declared", DECLARED)
@pytest.mark.parametrize("qexp,scale", [(-118, 2.0 ** 12), (-126, 2.0 ** 20), (-131, 2.0 ** 25)])
@pytest.mark.parametrize("d", [64, 128])
def test_tiny_queries_against_large_keys(qexp, scale, d, declared):
    """q down to bf16's subnormal numbers, |k| up to 2^108, scores of order 10: a
    row's largest value keeps its 8 bits whatever its exponent."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(-qexp)
    ctx, H, G = [40, 300, 5], 2, 4
    nb = 30
    pool = _random_pool(rng, nb, H, d)
    _set_k_scales(pool, 2.0 ** 101)
    bt = _tables(rng, ctx, nb)
    q, qt = _storage(rng.standard_normal((3, H * G, d)) * 2.0 ** qexp, "bf16")
    got = _decode(pk, qt, _dev(pool), bt, ctx, scale, torch.float32, 64, max_ctx=declared).double().cpu().numpy()
    ref = int8.paged_attention(q, pool, bt, ctx, scale)
    kd, vd = int8.dequant(pool, d)
    assert (np.abs(got - ref) <= _tolerance(oracle.to_f64(q), kd, vd, ctx, scale, False, ref)).all()


@pytest.mark.parametrize("declared", DECLARED)
@pytest.mark.parametrize("d", [64, 128])
def test_scores_of_zero_stay_zero_whatever_the_factors(d, declared):
    """Keys exactly orthogonal to a query have score 0 although the softmax scale,
    |q| and the K scale together pass fp32's range; one token whose score does fit
    takes the whole weight."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(d)
    ctx, H, G, nb = [50, 200], 1, 4, 20
    pool = _random_pool(rng, nb, H, d)
    byte = int8.record_positions(d)[0]
    pool[:, :, byte[:, ::2]] = 128                         # K is 0 in the even dims
    _set_k_scales(pool, 2.0 ** 102)
    bt = _tables(rng, ctx, nb)
    x = rng.uniform(0.5, 1, (2, H * G, d)) * 2.0 ** 60
    x[..., 1::2] = 0
    q, qt = _storage(x, "bf16")
    got = _decode(pk, qt, _dev(pool), bt, ctx, 2.0 ** 49, torch.float32, 64, max_ctx=declared).double().cpu().numpy()
    ref = int8.paged_attention(q, pool, bt, ctx, 2.0 ** 49)
    kd, vd = int8.dequant(pool, d)
    V = np.abs(vd).max()
    # the weights are exactly alike: the sums' roundings and the weights' 2^-22
    assert (np.abs(got - ref) <= V * 2 * ((max(ctx) / 16 + 8) * 2.0 ** -23 + 2.0 ** -22)).all()
    # 2^40 in dim 1 of q, 2^-19 of the largest (exact in f16), meets a code of 1 in token 33 of each
    # context and zeros elsewhere: a score of some 2^120 there, 2^139 times the token's code before
    x[..., 1] = 2.0 ** 40
    q, qt = _storage(x, "bf16")
    pool[:, :, byte[:, 1]] = 128
    for s in range(2):
        pool[bt[s, 2], :, byte[1, 1]] = 129
    got = _decode(pk, qt, _dev(pool), bt, ctx, 2.0 ** -22, torch.float32, 64, max_ctx=declared).double().cpu().numpy()
    _, vd = int8.dequant(pool, d)
    want = np.stack([vd[bt[s, 2], :, 1] for s in range(2)])                         # [2, H, d]
    assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -20).all()
