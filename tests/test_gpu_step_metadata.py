"""photon_build_step_metadata_device against the definition over plain lists
(oracle/fp4.py's step_metadata), its refusals on the device, and whole decode
steps over the 4-bit cache whose metadata never leaves the GPU."""
import numpy as np
import pytest

import oracle
from oracle import fp4
from tests.helpers import ensure_built
from tests.test_gpu_fp4 import _tolerance

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


class Dev:
    """Device buffers of a pool and a batch, with canaries behind the outputs."""

    def __init__(self, tables, stack, num_blocks, max_tokens):
        torch = _torch()
        B, W = tables.shape
        i32 = dict(dtype=torch.int32, device="cuda")
        self.tables = torch.from_numpy(np.ascontiguousarray(tables, np.int32)).cuda()
        self.free = torch.full((num_blocks,), -9, **i32)
        self.free[:len(stack)] = torch.tensor(stack, dtype=torch.int32)
        self.num_free = torch.tensor([len(stack)], **i32)
        M = max_tokens
        self.raw = [torch.full((M + 8,), -77, **i32), torch.full((M + 8,), -77, **i32),
                    torch.full((M + 8,), -77, dtype=torch.int64, device="cuda"), torch.full((B + 8,), -77, **i32)]
        self.seq, self.pos, self.slots = (x[:M] for x in self.raw[:3])
        self.lens = self.raw[3][:B]
        self.totals = torch.full((4,), -77, **i32)

    def step(self, pk, nc, nn, **kw):
        torch = _torch()
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
        pk.photon_build_step_metadata_device(t(nc), t(nn), self.tables, self.free, self.num_free, self.seq, self.pos,
                                             self.slots, self.lens, self.totals, **kw)
        torch.cuda.synchronize()

    def check(self, want):
        tables, stack, seq, pos, slots, ctx, status = want
        T = sum(p >= 0 for p in pos)
        assert self.totals.tolist() == [T, int(ctx.max()) if len(ctx) else 0, len(stack), status]
        assert np.array_equal(self.tables.cpu().numpy(), tables)
        assert self.num_free.item() == len(stack) and self.free[:len(stack)].tolist() == stack
        assert self.seq.tolist() == seq and self.pos.tolist() == pos and self.slots.tolist() == slots
        assert np.array_equal(self.lens.cpu().numpy(), ctx)
        for r in self.raw:
            assert (r[-8:] == -77).all()


def _start(rng, B, W, num_blocks, fill):
    """nc, tables and stack of a running batch whose rows hold ceil(nc / 16) blocks."""
    nc = np.where(rng.random(B) < fill, rng.integers(0, W * 8, B), 0).astype(np.int32)
    perm = [int(x) for x in rng.permutation(num_blocks)]
    tables = np.full((B, W), -1, np.int32)
    for s in range(B):
        for i in range(-(-int(nc[s]) // 16)):
            tables[s, i] = perm.pop()
    return nc, tables, perm


@pytest.mark.parametrize("B,W", [(1, 1), (1, 40), (7, 5), (64, 20), (1000, 6), (1025, 3), (3000, 4)])
@pytest.mark.parametrize("kind", ["decode", "mixed", "release", "idle"])
def test_steps_equal_the_definition(B, W, kind):
    pk = ensure_built()
    rng = np.random.default_rng(B + W)
    nb = B * W + 5
    nc, tables, stack = _start(rng, B, W, nb, 0.7)
    cap = W * 16
    if kind == "decode":
        nn = np.minimum(1, cap - nc)
    elif kind == "idle":
        nn = np.zeros(B, np.int32)
    else:
        nn = np.where(rng.random(B) < 0.3, 0, rng.integers(0, cap + 1, B))
        nn = np.minimum(nn, cap - nc)
    if kind == "release":
        nn = np.where(rng.random(B) < 0.5, -1 - rng.integers(0, 3, B), nn)
    M = int(np.maximum(nn, 0).sum()) + (0 if kind == "decode" else 13)
    dev = Dev(tables, stack, nb, M)
    pk.photon_device_errors()
    dev.step(pk, nc, nn)
    want = fp4.step_metadata(nc, nn, tables, stack, M, nb)
    assert want[-1] == 0
    dev.check(want)
    assert pk.photon_device_errors() == 0


def test_released_blocks_are_taken_again_in_the_same_step():
    pk = ensure_built()
    tables = np.array([[4, 5, 6], [-1, -1, -1], [2, -1, -1], [-1, -1, -1]], np.int32)
    nc, nn, stack = [48, 0, 3, 0], [-1, 30, -7, 40], [0, 1]
    dev = Dev(tables, stack, 7, 70)
    dev.step(pk, nc, nn)
    want = fp4.step_metadata(nc, nn, tables, stack, 70, 7)
    assert want[-1] == 0 and want[1] == [0, 1][:1] + want[1][1:]
    dev.check(want)


def test_many_steps_conserve_the_pool():
    pk = ensure_built()
    rng = np.random.default_rng(8)
    B, W, nb = 50, 12, 400
    nc, tables, stack = _start(rng, B, W, nb, 0.0)
    dev = Dev(tables, stack, nb, 2000)
    for step in range(60):
        nn = np.where(nc == 0, rng.integers(0, 60, B), 1).astype(np.int32)
        nn = np.where((nc > 0) & ((nc + 1 > W * 16) | (rng.random(B) < 0.05)), -1, nn)
        want = fp4.step_metadata(nc, nn, tables, stack, 2000, nb)
        dev.step(pk, nc, nn)
        dev.check(want)
        if want[-1] == 0:
            tables, stack, nc = want[0], want[1], want[5].astype(np.int32)
        else:                                   # pool exhausted: release the longest rows
            assert want[-1] == -5
            nn = np.where(nc >= np.median(nc[nc > 0]), -1, 0).astype(np.int32)
            want = fp4.step_metadata(nc, nn, tables, stack, 2000, nb)
            dev.step(pk, nc, nn)
            dev.check(want)
            tables, stack, nc = want[0], want[1], want[5].astype(np.int32)
        held = tables[tables >= 0].tolist()
        assert sorted(held + stack) == list(range(nb))
    pk.photon_device_errors()


@pytest.mark.parametrize("why", ["exhausted", "too many tokens", "row too short", "negative length", "overflow",
                                 "released row too long", "stack too high", "negative stack"])
def test_refused_steps_change_nothing(why):
    pk = ensure_built()
    B, W, nb, M = 5, 4, 12, 100
    tables = np.full((B, W), -1, np.int32)
    tables[0, :2] = [3, 4]
    nc, nn = np.array([20, 0, 0, 0, 0]), np.array([1, 30, 0, 5, 1])
    stack = [0, 1, 2, 5, 6, 7, 8, 9, 10, 11]
    status = -1
    if why == "exhausted":
        stack, status = [0, 1], -5
    elif why == "too many tokens":
        M = 36
    elif why == "row too short":
        nn[2] = 65
    elif why == "negative length":
        nc[4] = -1
    elif why == "overflow":
        nc[0] = 2 ** 31 - 1
    elif why == "released row too long":
        nc[3], nn[3] = 65, -1
    elif why == "stack too high":
        nb = 9
    dev = Dev(tables, stack[:nb], nb, M)
    if why == "stack too high":
        dev.num_free.fill_(10)
    if why == "negative stack":
        dev.num_free.fill_(-1)
    free0, count0 = dev.free.clone(), dev.num_free.clone()
    pk.photon_device_errors()
    dev.step(pk, nc, nn)
    assert pk.photon_device_errors() == pk.DEVERR_METADATA
    assert dev.totals.tolist() == [0, 0, int(count0), status]
    assert np.array_equal(dev.tables.cpu().numpy(), tables)
    assert _torch().equal(dev.free, free0) and _torch().equal(dev.num_free, count0)
    assert dev.seq.tolist() == [0] * M and dev.pos.tolist() == [-1] * M and dev.slots.tolist() == [-1] * M
    assert dev.lens.tolist() == [0] * B


def test_bad_block_ids_give_no_slot():
    pk = ensure_built()
    tables = np.array([[99, -1], [-4, -1], [2, -1]], np.int32)
    nc, nn = [3, 5, 15], [2, 1, 3]
    dev = Dev(tables, [0, 1, 50], 10, 8)
    pk.photon_device_errors()
    dev.step(pk, nc, nn)
    assert dev.slots.tolist() == [-1, -1, -1, 2 * 16 + 15, -1, -1, -1, -1]   # sequence 2 grows by block 50
    assert pk.photon_device_errors() == pk.DEVERR_BLOCK_RANGE


def test_no_sequences_and_no_tokens():
    torch = _torch()
    pk = ensure_built()
    dev = Dev(np.zeros((0, 3), np.int32), [1, 0], 2, 5)
    dev.step(pk, np.zeros(0), np.zeros(0))
    assert dev.totals.tolist() == [0, 0, 2, 0] and dev.slots.tolist() == [-1] * 5
    dev = Dev(np.array([[1, -1]], np.int32), [0], 2, 0)
    dev.step(pk, [16], [0])
    assert dev.totals.tolist() == [0, 16, 1, 0] and dev.lens.tolist() == [16]


def test_count_may_go_to_another_buffer():
    torch = _torch()
    pk = ensure_built()
    dev = Dev(np.full((1, 4), -1, np.int32), [3, 2, 1, 0], 4, 40)
    other = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(2):          # the same inputs give the same step
        dev.step(pk, [0], [33], num_free_out=other)
        assert other.item() == 1 and dev.num_free.item() == 4
        assert dev.tables.tolist() == [[0, 1, 2, -1]]


@pytest.mark.parametrize("M", [64, 5000])
def test_captured_decode_steps_over_the_4_bit_cache(M):
    """A whole step (metadata, 4-bit write, decode) captured once and replayed,
    the lengths advanced on the GPU: each step's output against the oracle on
    the pool's own codes, prompts admitted and a request released on the way."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(11)
    B, W, H, G, d, nb = 4, 8, 2, 4, 64, 40
    i32 = dict(dtype=torch.int32, device="cuda")
    nc, nn = torch.zeros(B, **i32), torch.zeros(B, **i32)
    k = torch.empty(M, H, d, dtype=torch.bfloat16, device="cuda")
    v, q = torch.empty_like(k), torch.empty(B, H * G, d, dtype=torch.bfloat16, device="cuda")
    dev = Dev(np.full((B, W), -1, np.int32), list(range(nb)), nb, M)
    pool = torch.randint(0, 256, (nb, H, 17 * d), dtype=torch.uint8, device="cuda")
    out = torch.empty(B, H * G, d, device="cuda")
    n = pk.photon_paged_attention_workspace_size(B, H * G, d, W * 16, 32)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def step():
        pk.photon_build_step_metadata_device(nc, nn, dev.tables, dev.free, dev.num_free, dev.seq, dev.pos, dev.slots,
                                             dev.lens, dev.totals)
        pk.photon_kv_cache_write_fp4(k, v, dev.pos, dev.slots, pool, 1e4)
        pk.photon_paged_attention_decode_fp4(q, pool, dev.tables, dev.lens, 0.125, out, W * 16, 32, ws)
        nc.copy_(dev.lens)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()                                    # nothing to do: every length is 0
    torch.cuda.synchronize()
    assert out.abs().max().item() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    tables, stack, host_nc = np.full((B, W), -1, np.int32), list(range(nb)), np.zeros(B, np.int32)
    for i in range(30):
        new = np.where(host_nc == 0, rng.integers(0, 16, B), 1).astype(np.int32)
        if i in (9, 20):
            new[i % B] = -1
        nn.copy_(torch.from_numpy(new))
        for t in (k, v, q):
            t.copy_(torch.from_numpy(rng.standard_normal(t.shape).astype(np.float32)))
        graph.replay()
        torch.cuda.synchronize()
        want = fp4.step_metadata(host_nc, new, tables, stack, M, nb)
        assert want[-1] == 0
        dev.check(want)
        tables, stack, host_nc = want[0], want[1], want[5].astype(np.int32)
        p = pool.cpu().numpy()
        ref = fp4.paged_attention(q.view(torch.int16).cpu().numpy().view(np.uint16), p,
                                  np.maximum(tables, 0), host_nc, 0.125)
        live = [(int(b), r) for s in range(B) for b, r in
                ((tables[s, x // 16], x % 16) for x in range(int(host_nc[s])))]
        kd, vd = fp4.dequant(p, d)
        kd, vd = (np.array([x[b, :, r] for b, r in live]) if live else np.zeros((1, H, d)) for x in (kd, vd))
        tol = _tolerance(q.double().cpu().numpy(), kd, vd, host_nc, 0.125, False, ref)
        assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    assert pk.photon_device_errors() == 0


def test_prefix_read_back_feeds_the_bf16_prefill():
    """A prefix written in 4 bits, read back to a bf16 staging pool, attended
    to by the prefill of the next chunk: the oracle's prefill on those values."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(21)
    H, G, d, nb = 2, 4, 64, 16
    prefix, chunk = 53, 20
    L = prefix + chunk
    bt = rng.permutation(nb)[:8].astype(np.int32)[None]
    pos = np.arange(L, dtype=np.int32)
    slots = bt[0, pos // 16].astype(np.int64) * 16 + pos % 16
    mk = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).bfloat16().cuda()
    k, v, q = mk(L, H, d), mk(L, H, d), mk(chunk, H * G, d)
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    pool = torch.zeros(nb, H, 17 * d, dtype=torch.uint8, device="cuda")
    pk.photon_kv_cache_write_fp4(k, v, cu(pos), cu(slots), pool, 1e4)
    kr, vr = torch.empty_like(k), torch.empty_like(v)
    pk.photon_kv_cache_read_fp4(pool, cu(slots), kr, vr)
    kc = torch.zeros(nb, H, 16, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    pk.photon_kv_cache_write(kr, vr, cu(pos), cu(slots), kc, vc, 1.0, "none")
    n = pk.photon_paged_attention_workspace_size(chunk, H * G, d, L, 32)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    out = torch.empty(chunk, H * G, d, device="cuda")
    pk.photon_paged_attention_prefill(q, cu(np.zeros(chunk, np.int32)), cu(pos[prefix:]), kc, vc, cu(bt), 0.125, out,
                                      L - 1, 32, ws)
    torch.cuda.synchronize()
    kd, vd = fp4.dequant(pool.cpu().numpy(), d)
    want = torch.from_numpy(kd[slots // 16, :, slots % 16]).bfloat16()
    assert torch.equal(kr.cpu(), want)
    bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)
    ref = oracle.paged_attention_prefill(bits(q), np.zeros(chunk, np.int32), pos[prefix:], bits(kc), bits(vc), bt,
                                         0.125)
    assert np.abs(out.cpu().numpy() - ref).max() <= 5e-3
    assert pk.photon_device_errors() == 0


@pytest.mark.parametrize("B", [1, 32, 33, 64, 65, 128, 200, 255, 256, 257, 1025])
@pytest.mark.parametrize("grown", [0, 3])
def test_a_step_that_takes_the_last_blocks(B, grown):
    """A step that leaves no block free, and one that needs none of an empty
    stack: the stack lies between other data, which stays as it was, and no
    value of which reaches a result."""
    torch = _torch()
    pk = ensure_built()
    grown = min(grown, B)
    nb = 2 * B + grown
    perm = np.random.default_rng(B).permutation(nb).astype(np.int32)
    nc = np.full(B, 20, np.int32)
    nc[:grown] = 32
    nn = np.ones(B, np.int32)
    tables = np.concatenate([perm[:2 * B].reshape(B, 2), np.full((B, 1), -1, np.int32)], 1)
    stack = [int(x) for x in perm[2 * B:]]
    dev = Dev(tables, stack, nb, B)
    room = torch.full((nb + 256,), 2 ** 30, dtype=torch.int32, device="cuda")
    room[128:128 + nb] = dev.free
    dev.free = room[128:128 + nb]
    pk.photon_device_errors()
    dev.step(pk, nc, nn)
    want = fp4.step_metadata(nc, nn, tables, stack, B, nb)
    assert want[-1] == 0 and want[1] == []
    dev.check(want)
    assert (room[:128] == 2 ** 30).all() and (room[128 + nb:] == 2 ** 30).all()
    assert pk.photon_device_errors() == 0


@pytest.mark.parametrize("B", [4, 300, 5000])
@pytest.mark.parametrize("bad", [-1, -7, "num_blocks", 2 ** 31 - 1])
@pytest.mark.parametrize("where", ["first", "last", "middle", "exhausted"])
def test_released_rows_with_foreign_blocks_are_refused(B, bad, where):
    """As photon_block_pool_free refuses such an id: nothing changes, whichever
    row and whichever CTA's share it lies in; the step without that row goes on."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(B)
    W, nb, M = 4, B * 4 + 3, 3 * B
    nc, tables, stack = _start(rng, B, W, nb, 1.0)
    nc = np.maximum(nc, 1)
    for s in range(B):
        if tables[s, 0] < 0:
            tables[s, 0] = stack.pop()
    nn = np.where(rng.random(B) < 0.5, -1, 1).astype(np.int32)
    nn[[0, B // 2, B - 1]] = -1
    row = {"first": 0, "last": B - 1, "middle": B // 2, "exhausted": B // 2}[where]
    if where == "exhausted":                     # too few blocks besides: the id is named first
        stack = stack[:0]
        nn[1] = 4 * 16 - nc[1]
        M = 70 + 3 * B
    good = tables.copy()
    at = int(rng.integers(0, -(-int(nc[row]) // 16)))
    tables[row, at] = nb if bad == "num_blocks" else bad
    dev = Dev(tables, stack, nb, M)
    free0 = dev.free.clone()
    pk.photon_device_errors()
    dev.step(pk, nc, nn)
    assert pk.photon_device_errors() == pk.DEVERR_METADATA | pk.DEVERR_BLOCK_RANGE
    assert dev.totals.tolist() == [0, 0, len(stack), -1]
    assert np.array_equal(dev.tables.cpu().numpy(), tables)
    assert torch.equal(dev.free[:len(stack)], free0[:len(stack)])
    want = fp4.step_metadata(nc, nn, tables, stack, M, nb)
    assert want[-1] == -1
    dev.check(want)
    nn[row] = 0                                   # the rest of the step, the row kept
    want = fp4.step_metadata(nc, nn, tables, stack, M, nb)
    dev.step(pk, nc, nn)
    dev.check(want)
    if want[-1] == 0:
        assert all(0 <= x < nb for x in want[1])
        assert pk.photon_device_errors() == 0
    tables = good
    dev = Dev(tables, stack, nb, M)               # and the sound row is released
    nn[row] = -1
    dev.step(pk, nc, nn)
    dev.check(fp4.step_metadata(nc, nn, tables, stack, M, nb))
    pk.photon_device_errors()


def test_lengths_survive_a_refused_step():
    """A captured step that advances its lengths on the GPU, only when the step
    was not refused: after one that ran out of blocks and one too long for its
    row, every row, block and length is there, and the decode goes on."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(14)
    B, W, H, G, d, nb, M = 3, 6, 2, 2, 64, 8, 100
    i32 = dict(dtype=torch.int32, device="cuda")
    nc, nn = torch.zeros(B, **i32), torch.zeros(B, **i32)
    k = torch.from_numpy(rng.standard_normal((M, H, d)).astype(np.float32)).bfloat16().cuda()
    v = torch.from_numpy(rng.standard_normal((M, H, d)).astype(np.float32)).bfloat16().cuda()
    q = torch.from_numpy(rng.standard_normal((B, H * G, d)).astype(np.float32)).bfloat16().cuda()
    dev = Dev(np.full((B, W), -1, np.int32), list(range(nb)), nb, M)
    pool = torch.zeros(nb, H, 17 * d, dtype=torch.uint8, device="cuda")
    out = torch.empty(B, H * G, d, device="cuda")
    ws = torch.empty(pk.photon_paged_attention_workspace_size(B, H * G, d, W * 16, 32), dtype=torch.uint8,
                     device="cuda")

    def step():
        pk.photon_build_step_metadata_device(nc, nn, dev.tables, dev.free, dev.num_free, dev.seq, dev.pos, dev.slots,
                                             dev.lens, dev.totals)
        pk.photon_kv_cache_write_fp4(k, v, dev.pos, dev.slots, pool, 1e4)
        pk.photon_paged_attention_decode_fp4(q, pool, dev.tables, dev.lens, 0.125, out, W * 16, 32, ws)
        torch.where(dev.totals[3] == 0, dev.lens, nc, out=nc)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    tables, stack, host_nc = np.full((B, W), -1, np.int32), list(range(nb)), np.zeros(B, np.int32)
    # 7 of 8 blocks; out of blocks; a row too long; one token each; the first released, the others grow
    plan = [([30, 40, 20], 0), ([3, 9, 20], -5), ([0, 57, 0], -1), ([1, 1, 1], 0), ([-1, 30, 5], 0), ([9, 1, 1], 0)]
    for new, status in plan:
        nn.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = fp4.step_metadata(host_nc, new, tables, stack, M, nb)
        assert want[-1] == status
        dev.check(want)
        if status:
            assert (out == 0).all() and np.array_equal(nc.cpu().numpy(), host_nc)
            continue
        tables, stack, host_nc = want[0], want[1], want[5].astype(np.int32)
        assert np.array_equal(nc.cpu().numpy(), host_nc)
        p = pool.cpu().numpy()
        ref = fp4.paged_attention(q.view(torch.int16).cpu().numpy().view(np.uint16), p, np.maximum(tables, 0),
                                  host_nc, 0.125)
        tol = _tolerance(q.double().cpu().numpy(), *fp4.dequant(p, d), host_nc, 0.125, False, ref)
        assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    held = tables[tables >= 0].tolist()
    assert sorted(held + stack) == list(range(nb))
    assert pk.photon_device_errors() == pk.DEVERR_METADATA


def test_the_order_in_which_released_blocks_are_taken_again():
    """The same step as test_released_blocks_are_taken_again_in_the_same_step,
    against the result written out: [0, 1] + [4, 5, 6] + [2] is popped from its end."""
    pk = ensure_built()
    tables = np.array([[4, 5, 6], [-1, -1, -1], [2, -1, -1], [-1, -1, -1]], np.int32)
    nc, nn = [48, 0, 3, 0], [-1, 30, -7, 40]
    dev = Dev(tables, [0, 1], 7, 70)
    dev.step(pk, nc, nn)
    assert dev.tables.tolist() == [[-1, -1, -1], [2, 6, -1], [-1, -1, -1], [5, 4, 1]]
    assert dev.free[:1].tolist() == [0] and dev.num_free.item() == 1
    assert dev.totals.tolist() == [70, 40, 1, 0] and dev.lens.tolist() == [0, 30, 0, 40]
    slots = [b * 16 + o for b in (2, 6) for o in range(16)][:30] + [b * 16 + o for b in (5, 4, 1) for o in range(16)][:40]
    assert dev.slots.tolist() == slots
    want = fp4.step_metadata(nc, nn, tables, [0, 1], 70, 7)
    assert np.array_equal(want[0], dev.tables.cpu().numpy()) and want[1] == [0]


@pytest.mark.parametrize("release", [False, True])
def test_as_many_sequences_as_a_step_takes(release):
    """16384 sequences: the sums fill a CTA's shared memory, sixteen to a thread."""
    pk = ensure_built()
    rng = np.random.default_rng(16)
    B, W = 16384, 3
    nb = B * W + 5
    nc, tables, stack = _start(rng, B, W, nb, 0.8)
    nn = np.minimum(rng.choice([0, 1, 1, 1, 20], B), W * 16 - nc)
    if release:
        nn = np.where(rng.random(B) < 0.4, -1, nn)
    M = int(np.maximum(nn, 0).sum()) + 3
    dev = Dev(tables, stack, nb, M)
    pk.photon_device_errors()
    dev.step(pk, nc, nn)
    want = fp4.step_metadata(nc, nn, tables, stack, M, nb)
    assert want[-1] == 0
    dev.check(want)
    assert pk.photon_device_errors() == 0


@pytest.mark.parametrize("B,H,G,d,first", [(64, 8, 4, 64, 200), (300, 2, 4, 128, 40), (2, 8, 2, 128, 900)])
@pytest.mark.parametrize("write", [False, True])
def test_back_to_back_steps_read_the_metadata_of_their_own_step(B, H, G, d, first, write):
    """Forty steps with no other kernel between them, streamed and captured:
    each decode reads lengths and tables early, and the buffers it reads are
    those that the decode two steps before it read with other contents."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(B)
    steps, W = 40, -(-(first + 60) // 16)
    nb = B * W
    i32 = dict(dtype=torch.int32, device="cuda")
    start = torch.from_numpy(rng.integers(first // 2, first, B).astype(np.int32)).cuda()
    perm = torch.from_numpy(rng.permutation(nb).astype(np.int32)).cuda()
    held = (start + 15) // 16
    col = torch.arange(W, device="cuda")[None]
    at = (held.cumsum(0) - held)[:, None] + col
    tables0 = torch.where(col < held[:, None], perm[at.clamp(max=nb - 1)], -1).int()
    used = int(held.sum())
    free0 = torch.zeros(nb, **i32)
    free0[:nb - used] = perm[used:]
    pool0 = torch.randint(0, 256, (nb, H, 17 * d), dtype=torch.uint8, device="cuda")
    byte, nib, sb = fp4.record_positions(d)
    for w in range(2):                                   # scales in (0, 2)
        pool0[:, :, sb[w].ravel() + 1] = 0x3E
    rows = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).bfloat16().cuda()
    k, v, q = rows(steps, B, H, d), rows(steps, B, H, d), rows(B, H * G, d)
    one = torch.ones(B, **i32)
    ws = torch.empty(max(1, pk.photon_paged_attention_workspace_size(B, H * G, d, W * 16, 64)), dtype=torch.uint8,
                     device="cuda")
    seq, pos = torch.empty(B, **i32), torch.empty(B, **i32)
    slots, totals = torch.empty(B, dtype=torch.int64, device="cuda"), torch.empty(4, **i32)
    tables, free, count, pool = tables0.clone(), free0.clone(), torch.empty(1, **i32), pool0.clone()
    lens = [torch.empty(B, **i32) for _ in range(2)]
    out = torch.empty(steps, B, H * G, d, device="cuda")

    def reset():
        tables.copy_(tables0), free.copy_(free0), pool.copy_(pool0), count.fill_(nb - used), lens[1].copy_(start)
        out.fill_(float("nan"))

    def chain(sync):
        for i in range(steps):
            pk.photon_build_step_metadata_device(lens[(i + 1) % 2], one, tables, free, count, seq, pos, slots,
                                                 lens[i % 2], totals)
            sync()
            if write:
                pk.photon_kv_cache_write_fp4(k[i], v[i], pos, slots, pool, 1e4)
                sync()
            pk.photon_paged_attention_decode_fp4(q, pool, tables, lens[i % 2], 0.1, out[i], W * 16, 64, ws)
            sync()

    pk.photon_device_errors()
    reset()
    chain(torch.cuda.synchronize)
    want = out.clone()
    assert torch.isfinite(want).all() and (want[1:] != want[:-1]).any(-1).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(lambda: None)
    for run in [lambda: chain(lambda: None)] * 5 + [graph.replay] * 5:
        reset()
        run()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert pk.photon_device_errors() == 0
