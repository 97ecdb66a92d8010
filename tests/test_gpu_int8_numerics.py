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
