"""The token loop of the step-metadata kernel (csrc/step_metadata.cu), checked
on the CPU through a direct model of its index arithmetic: which cells of the
block tables and of the free-block stack each lane addresses.

What the device code relies on: a warp takes `turns` rounds of 32 neighbouring
tokens, lanes past the last token repeat it, and only rounds below `turns`
load anything.  Every stack cell addressed then lies in [0, free + released),
whatever the stack holds, an empty one included."""
import numpy as np
import pytest

N = 4                      # rounds of a warp at most (kMetaBatch)


def _addresses(nc, nn, num_free, max_tokens, all_rounds=False):
    """(stack indices, table cells (s, b)) that the token loop loads for a step
    without released rows; all_rounds: the rounds from `turns` on load too."""
    nc, nn = np.asarray(nc, np.int64), np.asarray(nn, np.int64)
    B = len(nc)
    have, need = -(-nc // 16), -(-(nc + nn) // 16)
    tok, gro = np.cumsum(nn) - nn, np.cumsum(need - have) - (need - have)
    T = int(nn.sum())
    entries = max(max_tokens, B)
    ctas = 1
    while ctas * 2048 < entries and ctas < 16:
        ctas *= 2
    threads = ctas * (256 if entries <= 256 else 1024)
    turns = min(N, -(-T // threads))
    owner = lambda x: int(np.searchsorted(tok, x, side="right") - 1)
    stack, cells = [], []
    for warp in range(threads // 32):
        base = warp * 32 * turns
        while base < T:
            start = owner(base)
            for i in range(N):
                if i >= turns and not all_rounds:
                    continue
                for lane in range(32):
                    x = min(base + 32 * i + lane, T - 1)
                    s = owner(x) if i < turns else start
                    if i < turns and lane == 31:
                        start = s
                    b = int(nc[s] + x - tok[s]) // 16
                    if b < have[s]:
                        cells.append((s, b))
                    else:
                        stack.append(num_free - 1 - int(gro[s] + b - have[s]))
            base += threads * turns
    return stack, cells


def _full_pool(B):
    """Running sequences whose next token fits their last block, no block free."""
    return np.full(B, 20), np.ones(B, np.int64)


@pytest.mark.parametrize("B", [1, 31, 32, 33, 63, 64, 65, 100, 128, 200, 255, 256, 257, 1000, 1025])
def test_a_full_pool_reads_no_stack_cell(B):
    nc, nn = _full_pool(B)
    stack, cells = _addresses(nc, nn, 0, B)
    assert not stack and set(cells) == {(s, 1) for s in range(B)}


def test_rounds_past_the_last_would_leave_the_stack():
    """Why the rounds from `turns` on must not load: their lanes keep the
    warp's first owner, whose row their positions run past."""
    for B, lowest in ((64, -2), (256, -6)):
        stack, _ = _addresses(*_full_pool(B), 0, B, all_rounds=True)
        assert min(stack) == lowest


@pytest.mark.parametrize("seed", range(60))
def test_loads_stay_inside_the_tables_and_the_stack(seed):
    rng = np.random.default_rng(seed)
    B = int(rng.integers(1, 400))
    W = int(rng.integers(1, 20))
    nc = rng.integers(0, W * 16 + 1, B)
    nn = np.minimum(rng.choice([0, 1, 1, 1, 40, 300], B), W * 16 - nc)
    if seed % 3 == 0:
        nn = np.minimum(nn, (16 - nc % 16) % 16)        # nothing grows
    grown = int((-(-(nc + nn) // 16) - -(-nc // 16)).sum())
    free = grown if seed % 2 else grown + int(rng.integers(0, 5))
    stack, cells = _addresses(nc, nn, free, int(nn.sum()) + int(rng.integers(0, 3)))
    assert all(0 <= i < max(free, 0) for i in stack)
    assert all(0 <= b < W and b < -(-int(nc[s]) // 16) for s, b in cells)
    # every token's block is among what was loaded
    want = {(s, int(p) // 16) for s in range(B) for p in range(int(nc[s]), int(nc[s] + nn[s]))}
    assert {(s, b) for s, b in want if b * 16 < nc[s]} == set(cells)
    assert len(set(stack)) == sum(b * 16 >= nc[s] for s, b in want)
