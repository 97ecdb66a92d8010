"""Decode over the 4-bit cache at the lower end of q's range."""
import numpy as np
import pytest

import oracle
from oracle import fp4
from tests.helpers import ensure_built
from tests.test_gpu_fp4 import _decode, _dev, _random_pool, _storage, _tables, _tolerance, _torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("part", [64, 512])
@pytest.mark.parametrize("qexp,scale", [(-118, 2.0 ** 12), (-126, 2.0 ** 20), (-131, 2.0 ** 25)])
@pytest.mark.parametrize("d", [64, 128])
def test_tiny_queries_against_large_keys(qexp, scale, d, part):
    """q down to bf16's subnormal numbers, |k| of 2^104 and more, scores of order 10: a
    row's largest value keeps its 8 bits whatever its exponent."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(-qexp)
    ctx, H, G, nb = [40, 300, 5], 2, 4, 30
    pool = _random_pool(rng, nb, H, d)
    _, _, sb = fp4.record_positions(d)
    high = pool[:, :, sb[0] + 1].astype(np.int64) << 8 | pool[:, :, sb[0]]         # K scales' bf16 bits
    high = high + (105 << 7)                                                        # times 2^105
    pool[:, :, sb[0]], pool[:, :, sb[0] + 1] = high & 0xFF, high >> 8
    bt = _tables(rng, ctx, nb)
    q, qt = _storage(rng.standard_normal((3, H * G, d)) * 2.0 ** qexp, "bf16")
    got = _decode(pk, qt, _dev(pool), bt, ctx, scale, torch.float32, part).double().cpu().numpy()
    ref = fp4.paged_attention(q, pool, bt, ctx, scale)
    kd, vd = fp4.dequant(pool, d)
    assert (np.abs(got - ref) <= _tolerance(oracle.to_f64(q), kd, vd, ctx, scale, False, ref)).all()
