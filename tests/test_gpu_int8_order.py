"""8-bit writes whose tokens of one block do not stand together: reported, with
nothing but the blocks concerned touched; and lists that are in order: not reported."""
import numpy as np
import pytest

from tests.helpers import ensure_built
from tests.test_gpu_int8 import _dev, _runs, _torch

pytestmark = pytest.mark.gpu


def _write(slots, nb, H=1, d=64, norm=False):
    """The error bits of a write at `slots`, and the blocks that it changed."""
    torch = _torch()
    pk = ensure_built()
    T = len(slots)
    k = torch.randn(T, H, d, device="cuda").bfloat16()
    pool = torch.zeros(nb, H, 32 * d + 16, dtype=torch.uint8, device="cuda")
    pos, at = torch.zeros(T, dtype=torch.int32, device="cuda"), _dev(np.asarray(slots, np.int64))
    pk.photon_device_errors()
    if norm:
        w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
        pk.photon_qk_norm_rope_kv_cache_write_int8(None, None, k, k, pos, at, None, w, 1e-6, pool, 1e4)
    else:
        pk.photon_kv_cache_write_int8(k, k, pos, at, pool, 1e4)
    torch.cuda.synchronize()
    return pk.photon_device_errors(), set(torch.nonzero(pool.flatten(1).any(1)).flatten().tolist())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("norm", [False, True])
def test_short_calls_report_two_runs_of_a_block(d, norm):
    pk = ensure_built()
    bad = pk.DEVERR_BLOCK_ORDER
    singles = lambda n: (np.arange(n) * 16).astype(np.int64)
    assert _write([0, 16, 1], 4, 1, d, norm) == (bad, {0, 1})
    assert _write([5, -1, 6], 4, 1, d, norm) == (bad, {0})                     # a skipped token in between
    assert _write([5, 4 * 16, 6], 4, 2, d, norm) == (bad | pk.DEVERR_SLOT_RANGE, {0})
    for n, j in ((64, 63), (200, 199), (256, 255), (256, 130), (153, 152)):   # the first token's block, far behind
        s = singles(n)
        s[j] = 3
        assert _write(s, n, 1, d, norm)[0] == bad
    two = (singles(100)[None] + np.array([[4], [5]])).ravel()                  # two tokens of each of 100 sequences, token by token
    assert _write(two, 100, 1, d, norm)[0] == bad


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [300, 700, 1500, 2600, 6000])
def test_long_calls_report_two_runs_near_each_other(T, d):
    """At every distance with at most 15 tokens in between, wherever it falls in the tiles."""
    pk = ensure_built()
    rng = np.random.default_rng(T)
    for gap in range(1, 16):
        for at in rng.integers(0, T - gap - 1, 4).tolist() + [T - gap - 2]:
            slots = (np.arange(T) * 16).astype(np.int64)
            slots[at + gap + 1] = slots[at] + 1
            assert _write(slots, T, 1, d)[0] == pk.DEVERR_BLOCK_ORDER, (gap, at)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 17, 152, 153, 256, 257, 400, 3000])
def test_lists_in_order_report_nothing(T, d):
    """Runs of all lengths, whole prompts, tokens of a block in any order, skipped
    tokens between blocks, a slot that padding rows repeat."""
    rng = np.random.default_rng(T)
    for pick in ([1], [1, 2, 5, 16, 17], [T], [7], [16], [33, 1]):
        lens = []
        while sum(lens) < T:
            lens.append(min(int(rng.choice(pick)), T - sum(lens)))
        nb = sum(n // 16 + 2 for n in lens)
        slots = _runs(rng, nb, lens)
        assert _write(slots, nb, 1, d)[0] == 0
        start = [i for i in range(T) if i == 0 or slots[i] // 16 != slots[i - 1] // 16] + [T]
        mixed = np.concatenate([rng.permutation(slots[a:b]) for a, b in zip(start, start[1:])])
        assert _write(mixed, nb, 1, d)[0] == 0
        holes = np.concatenate([np.concatenate([slots[a:b], np.full(rng.integers(0, 3), -1)]) for a, b in zip(start, start[1:])])
        assert _write(holes, nb, 1, d)[0] == 0
    assert _write(np.concatenate([np.arange(T) * 16 + 16, np.full(40, 3)]), T + 1, 1, d)[0] == 0
