"""8-bit KV cache with a scale per block and head on the GPU: write, read and
decode against the definitions of oracle/int8.py, and the steps a program makes
of them."""
import numpy as np
import pytest

import oracle
import synth
from oracle import int8
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu

STYLES = {"neox": oracle.ROPE_NEOX, "gptj": oracle.ROPE_GPTJ, "none": oracle.ROPE_NONE}


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


def _random_pool(rng, nb, H, d, std=0.5):
    """Pool of random codes and scales of about std / 40, padding bytes of any kind."""
    pool = rng.integers(1, 256, (nb, H, 32 * d + 16), dtype=np.uint8)
    sc = np.abs(rng.standard_normal((nb, H, 2)) * std / 80 + std / 40).astype(np.float32)
    pool[:, :, -16:-8] = sc.view(np.uint8)
    return pool


def _tables(rng, ctx, nb, width=None):
    need = [-(-max(int(c), 0) // 16) for c in ctx]
    perm = rng.permutation(nb)
    W = max(1, max(need)) if width is None else width
    bt = np.full((len(ctx), W), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        bt[i, :n] = perm[at:at + n]
        at += n
    return bt


def _runs(rng, nb, lens):
    """Slots of runs of consecutive positions: each from an offset of its own over
    blocks of its own, in order."""
    perm, at, out = rng.permutation(nb), 0, []
    for n in lens:
        pos = int(rng.integers(0, 16)) + np.arange(n)
        out.append(perm[at + pos // 16] * 16 + pos % 16)
        at += pos[-1] // 16 + 1
    return np.concatenate(out).astype(np.int64)


# Declared longest contexts: the batch's own (short steps: clusters of CTAs), and one
# that makes the same batch a long step's, which is cut into pieces and merged.
DECLARED = [None, 40000]


def _decode(pk, q, pool, bt, ctx, scale, out_dtype, part, max_ctx=None, extra_rows=0):
    torch = _torch()
    B, Hq, d = q.shape
    if max_ctx is not None and bt.shape[1] * 16 < max_ctx:
        bt = np.concatenate([bt, np.full((B, -(-max_ctx // 16) - bt.shape[1]), -1, np.int32)], 1)
    mc = int(max(max(ctx), 1)) if max_ctx is None else max_ctx
    n = pk.photon_paged_attention_workspace_size(B, Hq, d, mc, part)
    ws = torch.randint(0, 256, (max(n, 1),), dtype=torch.uint8, device="cuda") if n else None
    out = torch.full((B + extra_rows, Hq, d), -7.0, dtype=out_dtype, device="cuda")
    pk.photon_paged_attention_decode_int8(q, pool, _dev(bt), _dev(np.asarray(ctx, np.int32)), scale, out[:B], mc, part, ws)
    torch.cuda.synchronize()
    return out


def _tolerance(q64, kd, vd, ctx, scale, out_bf16, ref):
    """Per output element.  Let V = max |v|.  A relative error e of a weight
    moves a weighted mean by at most 2 e V (numerator and denominator), one of
    the numerator's weights alone by e V.
      score: products of f16 by exact codes summed in fp32, at most d + 4
        roundings of 2^-24 (2^-23 where the tensor core truncates) of
        sum |q||k|, times the scales (three products more); ex2 within 2^-22
      weight times V scale in f16: 2^-12 (bf16 output) or f16 + remainder 2^-22
      sums over n tokens in fp32, one rounding per 16-token MMA: (n / 16 + 8) 2^-23
      output: half a step of the type, 2^-8 or 2^-24 of the value"""
    d = q64.shape[-1]
    V = np.abs(vd).max() if vd.size else 0.0
    qk = np.abs(q64).sum(-1).max() * np.abs(kd).max()
    e_score = abs(scale) * (d + 8) * 2.0 ** -23 * qk + 2.0 ** -22
    e_sum = (max(ctx) / 16 + 8) * 2.0 ** -23
    e_p = 2.0 ** -12 if out_bf16 else 2.0 ** -22
    return V * (2 * e_score + 2 * e_sum + e_p) + np.abs(ref) * (2.0 ** -8 if out_bf16 else 2.0 ** -24)


# ---- write -----------------------------------------------------------------------

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,lens", [(1, [1]), (3, [5]), (8, [1] * 20), (2, [37, 1, 16, 3]), (4, [16, 15, 17, 1, 2])])
def test_unrotated_codes_equal_the_oracle(H, lens, dtype, d):
    """Every byte of the pool: codes and scales of the written blocks bit for bit
    (kept rows among them), all other bytes as they were; slots -1 and past the
    pool write nothing and end a run."""
    pk = ensure_built()
    rng = np.random.default_rng(len(lens) * 10 + H + d)
    T, nb = sum(lens), sum(n // 16 + 2 for n in lens) + 2
    k, kt = _storage(rng.standard_normal((T, H, d)) * rng.lognormal(-1, 1, (T, 1, 1)), dtype)
    v, vt = _storage(rng.standard_normal((T, H, d)) * rng.lognormal(0, 2, (T, H, 1)), dtype)
    slots = _runs(rng, nb, lens)
    if T > 20:                                          # a token left out only where its block ends or begins
        cut = [t for t in range(1, T) if slots[t] % 16 == 0][:2]
        slots[cut] = [-1, nb * 16 + 3][:len(cut)]
    want = _random_pool(rng, nb, H, d)
    pool = _dev(want.copy())
    pos = np.zeros(T, np.int32)
    pk.photon_device_errors()
    pk.photon_kv_cache_write_int8(kt, vt, _dev(pos), _dev(slots), pool, 1e4, "none")
    eff = np.where(slots >= nb * 16, -1, slots)
    int8.write_rows(oracle.to_f64(k), eff, want, 0, d)
    int8.write_rows(oracle.to_f64(v), eff, want, 1, d)
    assert np.array_equal(pool.cpu().numpy(), want)
    assert pk.photon_device_errors() == (pk.DEVERR_SLOT_RANGE if (slots >= nb * 16).any() else 0)


@pytest.mark.parametrize("T,H,d,run", [(5003, 1, 64, 5003), (5003, 2, 128, 1), (3100, 1, 64, 7), (1300, 3, 128, 100), (700, 2, 64, 16)])
def test_long_batches_equal_the_oracle(T, H, d, run):
    """Tiles of 2 to 16 tokens: one run or sixteen per tile, runs that pass its
    end, a ragged last tile; values unrotated, so bit for bit."""
    pk = ensure_built()
    rng = np.random.default_rng(T + run)
    lens = [run] * (T // run) + ([T % run] if T % run else [])
    nb = sum(n // 16 + 2 for n in lens)
    k, kt = _storage(rng.standard_normal((T, H, d)), "bf16")
    v, vt = _storage(rng.standard_normal((T, H, d)) * 3, "bf16")
    slots = _runs(rng, nb, lens)
    want = _random_pool(rng, nb, H, d)
    pool = _dev(want.copy())
    pk.photon_kv_cache_write_int8(kt, vt, _dev(np.zeros(T, np.int32)), _dev(slots), pool, 1e6, "none")
    int8.write_rows(oracle.to_f64(k), slots, want, 0, d)
    int8.write_rows(oracle.to_f64(v), slots, want, 1, d)
    assert np.array_equal(pool.cpu().numpy(), want)


@pytest.mark.parametrize("H,d", [(8, 64), (3, 64), (2, 128), (5, 128)])
@pytest.mark.parametrize("pieces", [40, 900])
def test_runs_of_every_length_next_to_each_other(H, d, pieces):
    """Single tokens, chunks, whole blocks and long prompts mixed, with skipped
    tokens between them: every path of a tile beside the others, bit for bit."""
    pk = ensure_built()
    rng = np.random.default_rng(pieces + H)
    lens = rng.choice([1, 1, 1, 2, 5, 15, 16, 17, 33, 64], pieces).tolist()
    nb = sum(n // 16 + 2 for n in lens)
    slots, at = [], 0
    for n in lens:
        base = int(rng.choice([0, 0, rng.integers(0, 16)]))
        slots.append(at * 16 + base + np.arange(n))
        at += (base + n - 1) // 16 + 1
        if rng.random() < 0.2:
            slots.append(np.full(int(rng.integers(1, 20)), -1))
    slots = np.concatenate(slots).astype(np.int64)
    perm = rng.permutation(nb)
    slots = np.where(slots < 0, -1, perm[np.maximum(slots, 0) // 16] * 16 + slots % 16)
    T = len(slots)
    k, kt = _storage(rng.standard_normal((T, H, d)), "bf16")
    v, vt = _storage(rng.standard_normal((T, H, d)) * 2, "bf16")
    want = _random_pool(rng, nb, H, d)
    pool = _dev(want.copy())
    pk.photon_kv_cache_write_int8(kt, vt, _dev(np.zeros(T, np.int32)), _dev(slots), pool, 1e6, "none")
    int8.write_rows(oracle.to_f64(k), slots, want, 0, d)
    int8.write_rows(oracle.to_f64(v), slots, want, 1, d)
    assert np.array_equal(pool.cpu().numpy(), want)


def test_blocks_past_32_bits_of_the_pool():
    """Write, read and decode at the end of a pool of more than 2^32 bytes."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(8)
    d, H, nb = 128, 1, 1100000
    pool = torch.empty(nb, H, 32 * d + 16, dtype=torch.uint8, device="cuda")
    T = 40
    bt = (nb - 1 - np.arange(3))[None].astype(np.int32)
    slots = (bt[0, np.arange(T) // 16].astype(np.int64) * 16 + np.arange(T) % 16)
    k, kt = _storage(rng.standard_normal((T, H, d)), "bf16")
    pos = _dev(np.zeros(T, np.int32))
    pk.photon_kv_cache_write_int8(kt, kt, pos, _dev(slots), pool, 1e4, "none")
    small = np.zeros((3, H, 32 * d + 16), np.uint8)
    for w in range(2):
        int8.write_rows(oracle.to_f64(k), (2 - np.arange(T) // 16) * 16 + np.arange(T) % 16, small, w, d)
    assert np.array_equal(pool[nb - 3:].cpu().numpy()[..., :-8], small[..., :-8])
    kb, vb = (torch.empty(T, H, d, device="cuda") for _ in range(2))
    pk.photon_kv_cache_read_int8(pool, _dev(slots), kb, vb)
    want = int8.dequant(small, d)[0][2 - np.arange(T) // 16, :, np.arange(T) % 16].astype(np.float32)
    assert np.array_equal(kb.cpu().numpy(), want) and torch.equal(kb, vb)
    q, qt = _storage(rng.standard_normal((1, 4, d)), "bf16")
    for declared in DECLARED:
        got = _decode(pk, qt, pool, bt, [T], d ** -0.5, torch.float32, 64, max_ctx=declared).double().cpu().numpy()
        ref = int8.paged_attention(q, small, np.array([[2, 1, 0]], np.int32), [T], d ** -0.5)
        kd, vd = int8.dequant(small, d)
        assert (np.abs(got - ref) <= _tolerance(oracle.to_f64(q), kd, vd, [T], d ** -0.5, False, ref)).all()
    assert pk.photon_device_errors() == 0


def test_many_queries_beside_the_write():
    """So many query rows that they get a launch of their own: all of them, and
    the codes, as the bf16 write's norms give them."""
    torch = _torch()
    pk = ensure_built()
    gen = torch.Generator(device="cuda").manual_seed(3)
    T, H, Hq, d, nb = 8200, 2, 16, 128, 520
    mk = lambda h: torch.randn(T, h, d, generator=gen, device="cuda").bfloat16()
    q, k, v = mk(Hq), mk(H), mk(H)
    wq, wk = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda") for _ in range(2))
    wq, wk = wq.bfloat16(), wk.bfloat16()
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 3
    slots = torch.arange(T, device="cuda") + 5
    pool = torch.zeros(nb, H, 32 * d + 16, dtype=torch.uint8, device="cuda")
    kc, vc = (torch.zeros(nb, H, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q1, q2 = q.clone(), q.clone()
    pk.photon_qk_norm_rope_kv_cache_write_int8(q1, pos, k, v, pos, slots, wq, wk, 1e-6, pool, 1e6)
    pk.photon_qk_norm_rope_kv_cache_write(q2, pos, k, v, pos, slots, wq, wk, 1e-6, kc, vc, 1e6)
    assert torch.equal(q1, q2)
    kb, vb = (torch.empty(T, H, d, device="cuda") for _ in range(2))
    pk.photon_kv_cache_read_int8(pool, slots, kb, vb)
    sc = torch.from_numpy(int8.scales(pool.cpu().numpy()).copy()).cuda()[slots // 16]      # [T, H, 2]
    rows = kc[slots // 16, :, slots % 16].float()
    # half a step of the codes, and of the bf16 rows that they are compared with
    assert ((kb - rows).abs() <= 0.5 * sc[..., :1] * (1 + 2.0 ** -10) + rows.abs() * 2.0 ** -8).all()
    assert ((vb - v.float()).abs() <= 0.5 * sc[..., 1:] * (1 + 2.0 ** -10)).all()


def test_writes_on_another_stream_captured_and_replayed():
    """The same bytes on a side stream and from a graph, replayed with new rows;
    nothing is allocated."""
    torch = _torch()
    pk = ensure_built()
    gen = torch.Generator(device="cuda").manual_seed(4)
    T, H, d, nb = 70, 4, 64, 12
    k, v = (torch.randn(T, H, d, generator=gen, device="cuda") for _ in range(2))
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.arange(T, device="cuda") + 7
    start = _dev(_random_pool(np.random.default_rng(4), nb, H, d))
    call = lambda pool, **kw: pk.photon_kv_cache_write_int8(k, v, pos, slots, pool, 1e4, **kw)
    a, b, c = start.clone(), start.clone(), start.clone()
    call(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(b, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    call(c)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(c)
    for sign in (1, -1, 3):
        k.mul_(sign)
        c.copy_(start)
        g.replay()
        a.copy_(start)
        call(a)
        assert torch.equal(a, c)


def _check_rotated(got, before, y, slots, d, which):
    """Codes and scales of fp32-rotated rows against fp64 rows y.  A value is off
    by at most 2^-19 of its pair's length, which is at most sqrt 2 m: the scale
    by 2^-18 (relatively, two roundings of 2^-24 more), a quotient by
    127 * 2^-18.4 + 127 * 2^-23 < 127 * 2^-18 steps before its rounding.  With the
    scales that the GPU wrote, kept rows are exact."""
    nb, H = got.shape[:2]
    want = before.copy()
    int8.write_rows(y, slots, want, which, d)
    sg, sw = int8.scales(got)[..., which].astype(np.float64), int8.scales(want)[..., which].astype(np.float64)
    assert (np.abs(sg - sw) <= 2.0 ** -18 * sw).all()
    mine = before.copy()
    int8.write_rows(y, slots, mine, which, d, given=int8.scales(got)[..., which])
    byte = int8.record_positions(d)[which]
    cg, cm = got[:, :, byte].astype(int), mine[:, :, byte].astype(int)
    new = np.zeros((nb, 16), bool)
    live = slots >= 0
    new[slots[live] // 16, slots[live] % 16] = True
    assert np.array_equal(cg.transpose(0, 2, 1, 3)[~new], cm.transpose(0, 2, 1, 3)[~new])
    b, o = slots[live] // 16, slots[live] % 16
    quo = y[live] / np.where(sg > 0, sg, 1.0)[b][..., None]
    assert (np.abs(cg[b, :, o] - 128 - quo) <= 0.5 + 127 * 2.0 ** -18).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("style", ["neox", "gptj", "none"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("H,G,lens", [(1, 1, [1]), (3, 2, [5, 20]), (8, 2, [1] * 9), (2, 4, [400, 3, 330])])
def test_rotated_and_normalised_rows(H, G, lens, norm, style, dtype, d):
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(sum(lens) + d + G)
    T, nb = sum(lens), sum(n // 16 + 2 for n in lens) + 2
    k, kt = _storage(rng.standard_normal((T, H, d)) * 0.7, dtype)
    v, vt = _storage(rng.standard_normal((T, H, d)), dtype)
    q, qt = _storage(rng.standard_normal((T, H * G, d)), dtype)
    wk, wkt = _storage(1 + 0.3 * rng.standard_normal(d), dtype)
    wq, wqt = _storage(1 + 0.3 * rng.standard_normal(d), dtype)
    pos = rng.integers(0, 2 ** 20, T).astype(np.int32)
    slots = _runs(rng, nb, lens)
    before = _random_pool(rng, nb, H, d, std=1.0)
    pool = _dev(before.copy())
    if norm:
        pk.photon_qk_norm_rope_kv_cache_write_int8(qt, _dev(pos), kt, vt, _dev(pos), _dev(slots), wqt, wkt, 1e-6, pool, 5e5, style)
        yq = int8.norm_rope(q, wq, 1e-6, pos, 5e5, STYLES[style])
        allowed = np.abs(yq) * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) + int8.pair_length(yq, STYLES[style]) * 2.0 ** -19
        assert (np.abs(qt.double().cpu().numpy() - yq) <= allowed).all()
    else:
        pk.photon_kv_cache_write_int8(kt, vt, _dev(pos), _dev(slots), pool, 5e5, style)
    got = pool.cpu().numpy()
    _check_rotated(got, before, int8.norm_rope(k, wk if norm else None, 1e-6, pos, 5e5, STYLES[style]), slots, d, 0)
    want = before.copy()
    int8.write_rows(oracle.to_f64(v), slots, want, 1, d)
    at = int8.record_positions(d)[1]
    assert np.array_equal(got[:, :, at], want[:, :, at])
    assert np.array_equal(int8.scales(got)[..., 1], int8.scales(want)[..., 1])
    assert np.array_equal(got[:, :, -8:], before[:, :, -8:])          # the unused bytes
    untouched = np.setdiff1d(np.arange(nb), slots // 16)
    assert np.array_equal(got[untouched], before[untouched])
    assert pk.photon_device_errors() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_token_by_token_equals_the_oracle_and_stays_within_a_step(d):
    """Three sequences append 40 tokens, one a call, growing in magnitude, into
    blocks full of garbage: bit for bit the definition, and each value within
    one step of its block's last scale however often that grew."""
    pk = ensure_built()
    rng = np.random.default_rng(d)
    S, N, H = 3, 40, 2
    nb = 12
    want = rng.integers(0, 256, (nb, H, 32 * d + 16), dtype=np.uint8)
    pool = _dev(want.copy())
    tab = rng.permutation(nb)[:9].reshape(3, 3)
    size = np.stack([np.linspace(0.1, 2, N), np.geomspace(1e-4, 1e4, N), np.ones(N)])
    x = (rng.standard_normal((N, S, H, d)) * size.T[:, :, None, None]).astype(np.float32)
    for t in range(N):
        slots = (tab[:, t // 16] * 16 + t % 16).astype(np.int64)
        pk.photon_kv_cache_write_int8(_dev(x[t]), _dev(-x[t]), _dev(np.zeros(S, np.int32)), _dev(slots), pool, 1e4, "none")
        int8.write_rows(x[t].astype(np.float64), slots, want, 0, d)
        int8.write_rows(-x[t].astype(np.float64), slots, want, 1, d)
        assert np.array_equal(pool.cpu().numpy(), want), t
    kd, vd = int8.dequant(want[tab.ravel()], d)
    sc = int8.scales(want[tab.ravel()])
    for s in range(S):
        for t in range(N):
            b = 3 * s + t // 16
            for val, w, sign in ((kd, 0, 1), (vd, 1, -1)):
                assert (np.abs(val[b, :, t % 16] - sign * x[t, s]) <= sc[b, :, w][:, None] * (1 + 2.0 ** -20)).all()


@pytest.mark.parametrize("d", [64, 128])
def test_zeros_tiny_huge_and_non_finite_rows(d):
    """Blocks of zeros, of values below the least scale and of the largest
    floats; an infinity or a NaN makes its block's K (V) of that head NaN, kept
    NaN by later tokens and cleared by a new start."""
    pk = ensure_built()
    rng = np.random.default_rng(11)
    H, nb = 2, 8
    x = rng.standard_normal((7 * 16, H, d)).astype(np.float32)
    x[:16] = 0
    x[16:32] *= np.float32(2.0 ** -110)
    x[32:48] = np.float32(3.3e38) * rng.choice([-1, 1, 0.25], (16, H, d))
    x[50, 0, 3], x[70, 1, 9], x[90, 0, 0] = np.inf, np.nan, -np.inf
    slots = np.arange(7 * 16, dtype=np.int64)
    want = rng.integers(0, 256, (nb, H, 32 * d + 16), dtype=np.uint8)
    pool = _dev(want.copy())

    def write(x, slots):
        z = np.zeros(len(slots), np.int32)
        pk.photon_kv_cache_write_int8(_dev(x), _dev(x), _dev(z), _dev(slots), pool, 1e4, "none")
        for w in range(2):
            int8.write_rows(x.astype(np.float64), slots, want, w, d)
        g, o = pool.cpu().numpy(), want.copy()
        for a in (g, o):                                 # a NaN's bits are not compared
            s = np.ascontiguousarray(a[:, :, -16:-8]).view(np.float32)
            a[:, :, -16:-8] = np.where(np.isnan(s), np.float32(1), s).view(np.uint8)
        assert np.array_equal(g, o)
        assert np.array_equal(np.isnan(int8.scales(pool.cpu().numpy())), np.isnan(int8.scales(want)))

    write(x, slots)
    kd, _ = int8.dequant(pool.cpu().numpy(), d)
    assert (kd[0] == 0).all() and (kd[1] == 0).all() and np.isfinite(kd[2]).all()
    assert np.isnan(kd[3, 0]).all() and np.isfinite(kd[3, 1]).all() and np.isnan(kd[4, 1]).all() and np.isnan(kd[5, 0]).all()
    write(x[100:101], np.array([3 * 16 + 5]))            # a finite row into a NaN block
    assert np.isnan(int8.dequant(pool.cpu().numpy(), d)[0][3, 0]).all()
    write(x[100:101], np.array([3 * 16]))                # a new start
    kd, _ = int8.dequant(pool.cpu().numpy(), d)
    assert np.isfinite(kd[3]).all() and (kd[3, :, 1:] == 0).all()
    write(x[100:102], np.array([3, 7]))                  # into the block of zeros


def test_tokens_of_a_block_in_any_order():
    """A run's offsets need not rise; one that holds offset 0 anywhere starts the block anew."""
    pk = ensure_built()
    rng = np.random.default_rng(2)
    H, d, nb = 3, 64, 5
    off = rng.permutation(16)
    slots = np.concatenate([2 * 16 + off, 4 * 16 + off[off > 4]]).astype(np.int64)
    x, xt = _storage(rng.standard_normal((len(slots), H, d)), "bf16")
    want = _random_pool(rng, nb, H, d)
    pool = _dev(want.copy())
    pk.photon_kv_cache_write_int8(xt, xt, _dev(np.zeros(len(slots), np.int32)), _dev(slots), pool, 1e4, "none")
    for w in range(2):
        int8.write_rows(oracle.to_f64(x), slots, want, w, d)
    assert np.array_equal(pool.cpu().numpy(), want)


# ---- read ------------------------------------------------------------------------

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(1, 1), (33, 3), (200, 8), (5000, 2)])
def test_read_returns_the_rounded_products(T, H, dtype, d):
    """Bit for bit the fp32 product, rounded to the type; repeated slots; rows of
    slots -1 or past the pool left as they were."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(T + d)
    nb = 6
    pool = _random_pool(rng, nb, H, d)
    slots = rng.integers(0, nb * 16, T).astype(np.int64)
    skip = np.zeros(T, bool)
    if T > 1:
        skip[1::9] = True
        slots[1::18], slots[10::18] = -1, nb * 16
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    k, v = (torch.full((T, H, d), -3.0, dtype=dt, device="cuda") for _ in range(2))
    pk.photon_device_errors()
    pk.photon_kv_cache_read_int8(_dev(pool), _dev(slots), k, v)
    torch.cuda.synchronize()
    for got, val in zip((k, v), int8.dequant(pool, d)):
        want = val[np.clip(slots, 0, nb * 16 - 1) // 16, :, np.clip(slots, 0, nb * 16 - 1) % 16]
        want = torch.from_numpy(np.where(skip[:, None, None], -3.0, want)).float().to(dt)
        assert torch.equal(got.cpu(), want)
    assert pk.photon_device_errors() == (pk.DEVERR_SLOT_RANGE if (slots >= nb * 16).any() else 0)


def test_read_longer_than_one_grid():
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(9)
    d, nb, T = 64, 3, 64 * 65535 + 77
    pool = _random_pool(rng, nb, 1, d)
    slots = torch.randint(0, nb * 16, (T,), generator=torch.Generator().manual_seed(1)).cuda()
    k, v = (torch.empty(T, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pk.photon_kv_cache_read_int8(_dev(pool), slots, k, v)
    for got, val in zip((k, v), int8.dequant(pool, d)):
        rows = torch.from_numpy(val[:, 0].reshape(nb * 16, d)).float().bfloat16().cuda()
        assert torch.equal(got[:, 0], rows[slots])


# ---- decode ----------------------------------------------------------------------

CONTEXTS = [([1, 17, 600, 1500, 33, 0], 256), ([3000, 9, 700, 0, 16], 512),
            ([16, 31, 32, 33, 47, 48, 49, 63, 64, 65, 511, 512, 513, 15], 64), ([1024], 32), ([5], 512), ([130, 0], 16),
            ([2500, 300], 4096)]


@pytest.mark.parametrize("declared", DECLARED)
@pytest.mark.parametrize("ctx,part", CONTEXTS)
@pytest.mark.parametrize("H,G", [(8, 1), (8, 2), (8, 4), (4, 8), (1, 4), (3, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_decode_matches_the_oracle(ctx, part, H, G, d, out, declared):
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(sum(ctx) + H * G + d)
    nb = sum(-(-c // 16) for c in ctx) + 3
    pool = _random_pool(rng, nb, H, d)
    bt = _tables(rng, ctx, nb)
    q, qt = _storage(rng.standard_normal((len(ctx), H * G, d)), "bf16")
    scale = d ** -0.5
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    got = _decode(pk, qt, _dev(pool), bt, ctx, scale, dt, part, max_ctx=declared, extra_rows=2)
    ref = int8.paged_attention(q, pool, bt, ctx, scale)
    assert (got[len(ctx):] == -7.0).all()                  # rows behind the batch
    got = got[:len(ctx)].double().cpu().numpy()
    kd, vd = int8.dequant(pool, d)
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= _tolerance(oracle.to_f64(q), kd, vd, ctx, scale, out == "bf16", ref)).all()
    for s, c in enumerate(ctx):
        if c == 0:
            assert (got[s] == 0).all()
    assert pk.photon_device_errors() == 0


@pytest.mark.parametrize("declared", DECLARED)
@pytest.mark.parametrize("qexp,vexp,scale", [(0, 0, -0.3), (100, 0, 2.0 ** -103), (-100, 0, 2.0 ** 97), (120, 0, 0.0), (123, 0, 2.0 ** -126),
                                             (0, 60, 0.125), (0, -100, 0.125), (0, 105, 0.125), (3, -60, -0.01), (-130, 0, 0.5)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_is_scale_free(qexp, vexp, scale, d, declared):
    """q and V scales of any magnitude, blocks of zeros, a negative or zero softmax scale."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(7)
    ctx, H, G = [300, 40, 1], 2, 4
    nb = 30
    pool = _random_pool(rng, nb, H, d)
    sc = int8.scales(pool).copy()
    sc[..., 1] = sc[..., 1] * 2.0 ** vexp * (rng.random(sc.shape[:2]) < 0.8)
    pool[:, :, -16:-8] = sc.astype(np.float32).view(np.uint8)
    bt = _tables(rng, ctx, nb)
    q, qt = _storage(rng.standard_normal((3, H * G, d)) * 2.0 ** qexp, "bf16")
    got = _decode(pk, qt, _dev(pool), bt, ctx, scale, torch.float32, 64, max_ctx=declared).double().cpu().numpy()
    ref = int8.paged_attention(q, pool, bt, ctx, float(np.float32(scale)))
    kd, vd = int8.dequant(pool, d)
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= _tolerance(oracle.to_f64(q), kd, vd, ctx, scale, False, ref) + 2.0 ** -149).all()


@pytest.mark.parametrize("declared", DECLARED)
@pytest.mark.parametrize("jump", [-40, 40, 100])
def test_decode_keeps_earlier_tokens_when_v_scales_jump(jump, declared):
    """V of the later half of a context 2^jump times the earlier one's, whose
    weights dominate: nothing of either half is lost beyond the tolerance."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(17)
    d, H, G, ctx = 64, 1, 4, [640, 96]
    nb = 50
    pool = _random_pool(rng, nb, H, d)
    bt = _tables(rng, ctx, nb)
    sc = int8.scales(pool).copy()
    for s, c in enumerate(ctx):
        sc[bt[s, c // 32:c // 16], :, 1] *= np.float32(2.0 ** jump)
    pool[:, :, -16:-8] = sc.view(np.uint8)
    q, qt = _storage(rng.standard_normal((2, H * G, d)), "bf16")
    for part in (64, 1024):
        got = _decode(pk, qt, _dev(pool), bt, ctx, 0.125, torch.float32, part, max_ctx=declared).double().cpu().numpy()
        ref = int8.paged_attention(q, pool, bt, ctx, 0.125)
        kd, vd = int8.dequant(pool, d)
        assert (np.abs(got - ref) <= _tolerance(oracle.to_f64(q), kd, vd, ctx, 0.125, False, ref)).all()


@pytest.mark.parametrize("declared", DECLARED)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("part", [32, 512])
def test_decode_ignores_everything_past_the_context(d, part, declared):
    """Any bytes in a page's tail rows and NaN scales in unused blocks leave every
    bit of the output as it was."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(d + part)
    ctx, H, G = [1, 15, 37, 200, 449, 64], 2, 4
    nb = 80
    pool = _random_pool(rng, nb, H, d)
    bt = _tables(rng, ctx, nb, width=32)
    _, qt = _storage(rng.standard_normal((len(ctx), H * G, d)), "bf16")
    a = _decode(pk, qt, _dev(pool), bt, ctx, 0.2, torch.float32, part, max_ctx=declared)
    byte = int8.record_positions(d)
    used = np.zeros((nb, 16), bool)
    for s, c in enumerate(ctx):
        for p in range(c):
            used[bt[s, p // 16], p % 16] = True
    for b, r in zip(*np.nonzero(~used)):
        for w in range(2):
            pool[b][:, byte[w, r]] = rng.integers(0, 256, (H, d))
    pool[~used.any(1), :, -16:-8] = np.array([np.nan, np.inf], np.float32).view(np.uint8)
    b_ = _decode(pk, qt, _dev(pool), bt, ctx, 0.2, torch.float32, part, max_ctx=declared)
    assert torch.equal(a, b_) and torch.isfinite(a).all()
    assert pk.photon_device_errors() == 0


@pytest.mark.parametrize("declared", DECLARED)
@pytest.mark.parametrize("part", [32, 1024])
@pytest.mark.parametrize("which", [0, 1])
def test_a_nan_block_makes_its_readers_nan(which, part, declared):
    """Every head over a block with a NaN scale, in the sequences whose contexts
    reach it, and no other row."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(part)
    d, H, G, ctx = 64, 2, 4, [100, 100, 33, 7]
    nb = 20
    pool = _random_pool(rng, nb, H, d)
    bt = _tables(rng, ctx, nb)
    pool[bt[1, 3], 1, -16:-8].view(np.float32)[which] = np.nan
    _, qt = _storage(rng.standard_normal((4, H * G, d)), "bf16")
    for dt in (torch.bfloat16, torch.float32):
        got = _decode(pk, qt, _dev(pool), bt, ctx, 0.125, dt, part, max_ctx=declared)
        nan = torch.isnan(got).cpu().numpy()
        assert nan[1, G:].all() and nan.sum() == G * d


@pytest.mark.parametrize("declared", DECLARED)
def test_bad_block_ids_and_lengths_are_reported_and_skipped(declared):
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(3)
    d, H, G, nb = 64, 2, 2, 40
    pool = _random_pool(rng, nb, H, d)
    for part in (32, 512):
        ctx = [200, 90, 48]
        bt = _tables(rng, ctx, nb)
        bt[0, 3], bt[0, 7], bt[1, 0], bt[2, :3] = -1, nb, 2 ** 31 - 1, -5
        _, qt = _storage(rng.standard_normal((3, H * G, d)), "bf16")
        pk.photon_device_errors()
        got = _decode(pk, qt, _dev(pool), bt, ctx, 0.125, torch.float32, part, max_ctx=declared)
        assert pk.photon_device_errors() == pk.DEVERR_BLOCK_RANGE
        assert torch.isfinite(got).all() and (got[2] == 0).all()
        # what is left: the tokens of the good pages
        for s in (0, 1):
            good = [i for i in range(-(-ctx[s] // 16)) if 0 <= bt[s, i] < nb]
            kd, vd = (x[bt[s, good]] for x in int8.dequant(pool, d))
            keep = np.concatenate([i * 16 + np.arange(16) < ctx[s] for i in good])
            q64 = qt[s].double().cpu().numpy()
            for h in range(H * G):
                kk, vv = (x[:, h // G].reshape(-1, d)[keep] for x in (kd, vd))
                p = np.exp(0.125 * kk @ q64[h] - (0.125 * kk @ q64[h]).max())
                ref = p @ vv / p.sum()
                assert np.abs(got[s, h].double().cpu().numpy() - ref).max() <= 1e-4
    # a length past the declared one is cut to it
    bt = _tables(rng, [64], nb)
    a = _decode(pk, qt[:1].contiguous(), _dev(pool), bt, [64], 0.125, torch.float32, 32, max_ctx=64)
    b = _decode(pk, qt[:1].contiguous(), _dev(pool), bt, [5000], 0.125, torch.float32, 32, max_ctx=64)
    assert torch.equal(a, b) and pk.photon_device_errors() == pk.DEVERR_CONTEXT_RANGE


@pytest.mark.parametrize("B,lo,hi,H,G,d,part,out", [
    (96, 256, 6000, 8, 4, 64, 512, "bf16"), (48, 16, 3000, 8, 2, 128, 128, "bf16"), (40, 500, 500, 8, 4, 64, 512, "bf16"),
    (60, 100, 1000, 8, 4, 128, 512, "bf16"), (3, 20000, 20000, 4, 8, 128, 256, "f32"), (1, 30000, 30000, 1, 8, 64, 512, "f32"),
    (300, 1, 200, 8, 1, 64, 64, "f32"), (300, 1, 200, 8, 2, 128, 64, "bf16"), (20, 100, 900, 8, 4, 64, 64, "bf16"), (30, 300, 900, 8, 8, 128, 128, "f32"),
    (1, 4096, 4096, 8, 4, 64, 64, "bf16"), (2, 5000, 5000, 1, 8, 128, 64, "f32"), (1, 8192, 8192, 4, 4, 64, 8192, "bf16"), (200, 2000, 9000, 2, 1, 64, 16384, "bf16"), (64, 5000, 8000, 8, 4, 64, 512, "f32"), (160, 3000, 5000, 4, 2, 128, 512, "bf16")])
def test_decode_grids(B, lo, hi, H, G, d, part, out):
    """Batches that take each of the launch shapes, against attention over the
    dequantised values in fp64 on the GPU; twice the same bits."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(B + hi)
    ctx = rng.integers(lo, hi + 1, B)
    if B > 2:
        ctx[B // 2], ctx[B // 3] = 0, 1
    nb = int(sum(-(-c // 16) for c in ctx)) + 2
    bank = _random_pool(rng, 64, H, d)
    pick = rng.integers(0, 64, nb)
    pool = _dev(bank)[_dev(pick)].contiguous()
    bt = _tables(rng, ctx, nb)
    _, qt = _storage(rng.standard_normal((B, H * G, d)), "bf16")
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    got = _decode(pk, qt, pool, bt, ctx, d ** -0.5, dt, part)
    assert torch.equal(got, _decode(pk, qt, pool, bt, ctx, d ** -0.5, dt, part))
    kd, vd = (_dev(x) for x in int8.dequant(bank, d))
    tab = _dev(pick)[_dev(np.maximum(bt, 0)).long()]
    ref = torch.zeros(B, H * G, d, dtype=torch.float64, device="cuda")
    for s in range(B):
        if ctx[s]:
            n = -(-int(ctx[s]) // 16)
            k, v = (x[tab[s, :n]].transpose(0, 1).flatten(1, 2)[:, :int(ctx[s])] for x in (kd, vd))
            p = torch.softmax(qt[s].double().view(H, G, d) @ k.mT * d ** -0.5, -1)
            ref[s] = (p @ v).view(H * G, d)
    ref = ref.cpu().numpy()
    allowed = _tolerance(qt.double().cpu().numpy(), kd.cpu().numpy(), vd.cpu().numpy(), ctx, d ** -0.5, out == "bf16", ref)
    assert (np.abs(got.double().cpu().numpy() - ref) <= allowed).all()
    assert pk.photon_device_errors() == 0


def test_two_streams_with_their_own_workspaces():
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(21)
    d, H, G = 128, 4, 2
    ctx = [[900, 40, 700], [33, 2000, 1]]
    nb = 260
    pool = _dev(_random_pool(rng, nb, H, d))
    sets = []
    for c in ctx:
        _, qt = _storage(rng.standard_normal((3, H * G, d)), "bf16")
        n = pk.photon_paged_attention_workspace_size(3, H * G, d, 2048, 128)
        sets.append((qt, _dev(_tables(rng, c, nb, width=128)), _dev(np.array(c, np.int32)), torch.cuda.Stream(),
                     [torch.zeros(3, H * G, d, device="cuda") for _ in range(6)],
                     torch.empty(n, dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    for i in range(6):
        for qt, bt, cl, st, outs, ws in sets:
            pk.photon_paged_attention_decode_int8(qt, pool, bt, cl, 0.1, outs[i], 2048, 128, ws, stream=st)
    torch.cuda.synchronize()
    for qt, bt, cl, st, outs, ws in sets:
        pk.photon_paged_attention_decode_int8(qt, pool, bt, cl, 0.1, outs[0], 2048, 128, ws)
        assert all(torch.equal(outs[0], o) for o in outs[1:])


# ---- as a program uses them -----------------------------------------------------

@pytest.mark.parametrize("d,H,G", [(64, 4, 4), (128, 2, 2)])
def test_prompts_then_captured_decode_steps(d, H, G):
    """Metadata on the GPU, prompts through the normalising 8-bit write, their
    prefix read back for a bf16 prefill, then a captured step (metadata, write,
    decode) replayed over block borders with rows released and admitted: every
    output against fp64 attention over the pool as it then stands."""
    torch = _torch()
    pk = ensure_built()
    gen = torch.Generator(device="cuda").manual_seed(d)
    B, W, nb, M, part, eps, theta = 5, 12, 64, 512, 64, 1e-6, 1e6
    i32 = dict(dtype=torch.int32, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    pool = torch.randint(0, 256, (nb, H, 32 * d + 16), dtype=torch.uint8, generator=gen, device="cuda")
    tables = torch.full((B, W), -1, **i32)
    free, num_free = torch.randperm(nb, generator=gen, device="cuda").int(), torch.full((1,), nb, **i32)
    nc, nn = torch.zeros(B, **i32), torch.tensor([37, 1, 16, 90, 15], **i32)
    seq, pos = torch.zeros(M, **i32), torch.zeros(M, **i32)
    slots = torch.zeros(M, dtype=torch.int64, device="cuda")
    lens, totals = torch.zeros(B, **i32), torch.zeros(4, **i32)
    wq, wk = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda") for _ in range(2))
    wq, wk = wq.bfloat16(), wk.bfloat16()
    n = pk.photon_paged_attention_workspace_size(B, H * G, d, W * 16, part)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def rows(T):
        return [torch.randn(T, h, d, generator=gen, device="cuda").bfloat16() for h in (H * G, H, H)]

    def expect(q, at, contexts):
        """fp64 attention of q[i] over the first contexts[i] tokens of row at[i]."""
        kd, vd = (_dev(x) for x in int8.dequant(pool.cpu().numpy(), d))
        out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        for i, (s, c) in enumerate(zip(at, contexts)):
            if c:
                t = tables[s, :-(-c // 16)].long()
                k, v = (x[t].transpose(0, 1).flatten(1, 2)[:, :c] for x in (kd, vd))
                out[i] = (torch.softmax(q[i].double().view(H, G, d) @ k.mT * d ** -0.5, -1) @ v).view(H * G, d)
        return out, kd, vd

    # prompts: written in 8 bits, then read back into bf16 pages that a prefill attends to
    pk.photon_build_step_metadata_device(nc, nn, tables, free, num_free, seq, pos, slots, lens, totals)
    T = int(totals[0])
    q, k, v = rows(M)
    pk.photon_qk_norm_rope_kv_cache_write_int8(q, pos.clamp(min=0), k, v, pos, slots, wq, wk, eps, pool, theta)
    kb, vb = (torch.zeros(M, H, d, **bf) for _ in range(2))
    pk.photon_kv_cache_read_int8(pool, slots, kb, vb)
    kc, vc = (torch.zeros(nb, H, 16, d, **bf) for _ in range(2))
    pk.photon_kv_cache_write(kb, vb, pos, slots, kc, vc, theta, "none")
    out = torch.zeros(M, H * G, d, device="cuda")
    wp = torch.empty(pk.photon_paged_attention_workspace_size(M, H * G, d, W * 16, 512), dtype=torch.uint8, device="cuda")
    pk.photon_paged_attention_prefill(q, seq, pos, kc, vc, tables, d ** -0.5, out, W * 16 - 1, 512, wp)
    want, kd, vd = expect(q[:T], seq[:T].tolist(), (pos[:T] + 1).tolist())
    # the prefill saw bf16 roundings of the values (2^-8 of K moves a score by 2^-8 sum |q||k|, V by 2^-8)
    kmax, vmax = kd[tables[tables >= 0].long()].abs().max().item(), vd[tables[tables >= 0].long()].abs().max().item()
    e = d ** -0.5 * q[:T].double().abs().sum(-1).max().item() * kmax * 2.0 ** -8
    assert (out[:T].double() - want).abs().max().item() <= vmax * (np.expm1(2 * e) + 2.0 ** -8 + 2.0 ** -10)

    nc.copy_(lens)
    qd, kd_, vd_ = rows(B)
    out = torch.zeros(B, H * G, d, device="cuda")
    dseq, dpos = torch.zeros(B, **i32), torch.zeros(B, **i32)
    dslots = torch.zeros(B, dtype=torch.int64, device="cuda")

    def step():
        pk.photon_build_step_metadata_device(nc, nn, tables, free, num_free, dseq, dpos, dslots, lens, totals)
        pk.photon_qk_norm_rope_kv_cache_write_int8(qd, dpos.clamp_(min=0), kd_, vd_, dpos, dslots, wq, wk, eps, pool, theta)
        pk.photon_paged_attention_decode_int8(qd, pool, tables, lens, d ** -0.5, out, W * 16, part, ws)
        nc.copy_(torch.where(totals[3] == 0, lens, nc))

    state = [t.clone() for t in (nc, tables, free, num_free, pool, qd)]
    nn.fill_(1)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(g):
        step()
    for t, s in zip((nc, tables, free, num_free, pool, qd), state):
        t.copy_(s)
    pk.photon_device_errors()
    for i in range(22):
        nn.fill_(1)
        if i == 7:
            nn[1] = -1                       # released; its blocks may be handed out again
        if i == 8:
            nn[1] = 1                        # admitted again from nothing
        tokens = [s for s in range(B) if int(nn[s]) > 0]
        new = rows(B)
        for t, x in zip((qd, kd_, vd_), new):
            t.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert int(totals[3]) == 0 and pk.photon_device_errors() == 0
        contexts = lens.tolist()
        # the write normalises the rows of the step's tokens, which stand first in the list
        want, kd, vd = expect(qd, range(B), contexts)
        used = torch.unique(tables[tables >= 0].long())
        allowed = _tolerance(qd.double().cpu().numpy(), kd[used].cpu().numpy(), vd[used].cpu().numpy(), contexts, d ** -0.5,
                             False, want.cpu().numpy())
        assert (np.abs(out.double().cpu().numpy() - want.cpu().numpy()) <= allowed).all(), i
        assert len(tokens) == int(totals[0])


def test_refusals():
    torch = _torch()
    pk = ensure_built()
    T, H, d = 4, 2, 64
    f = dict(dtype=torch.bfloat16, device="cuda")
    q, k, v, w = torch.zeros(T, 4, d, **f), torch.zeros(T, H, d, **f), torch.zeros(T, H, d, **f), torch.zeros(d, **f)
    pos, slots = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.arange(T, device="cuda")
    pool = torch.zeros(2, H, 32 * d + 16, dtype=torch.uint8, device="cuda")
    bt, cl = torch.zeros(T, 2, dtype=torch.int32, device="cuda"), torch.ones(T, dtype=torch.int32, device="cuda")
    calls = {
        "write": (pk.photon_kv_cache_write_int8, dict(k=k, v=v, positions=pos, slot_mapping=slots, kv_cache=pool, rope_theta=1e4)),
        "norm": (pk.photon_qk_norm_rope_kv_cache_write_int8,
                 dict(q=q, q_positions=pos, k=k, v=v, positions=pos, slot_mapping=slots, q_weight=w, k_weight=w, eps=1e-6,
                      kv_cache=pool, rope_theta=1e4)),
        "read": (pk.photon_kv_cache_read_int8, dict(kv_cache=pool, slot_mapping=slots, k=k, v=v)),
        "decode": (pk.photon_paged_attention_decode_int8,
                   dict(q=q, kv_cache=pool, block_tables=bt, context_lens=cl, scale=0.1, out=torch.zeros_like(q), max_context_len=32)),
    }
    bad = {
        "write": [dict(v=v[:1]), dict(kv_cache=pool[..., :-16].contiguous()), dict(positions=pos.long()), dict(slot_mapping=slots.int()),
                  dict(k=k.half(), v=v.half()), dict(k=k.cpu()), dict(kv_cache=pool.cpu()), dict(rope_theta=0.0), dict(rope_style=5),
                  dict(k=k[..., :32].contiguous(), v=v[..., :32].contiguous()), dict(kv_cache=pool.transpose(0, 1))],
        "norm": [dict(eps=0.0), dict(q_weight=w.float()), dict(k_weight=w[:8]), dict(q=q.float()), dict(q_positions=pos[:2])],
        "read": [dict(v=v.float()), dict(slot_mapping=slots.int()), dict(kv_cache=pool[:, :1].contiguous())],
        "decode": [dict(q=q.float()), dict(out=torch.zeros(T, 4, d, dtype=torch.float16, device="cuda")), dict(block_tables=bt.long()),
                   dict(context_lens=cl[:2]), dict(max_context_len=64), dict(partition_size=24), dict(partition_size=16),
                   dict(scale=float("nan")), dict(kv_cache=pool[:, :1].contiguous(), q=q[:, :3].contiguous(), out=torch.zeros(T, 3, d, **f))],
    }
    for name, (f_, args) in calls.items():
        f_(**args)
        for kw in bad[name]:
            with pytest.raises((TypeError, ValueError, KeyError, pk.PhotonError)):
                f_(**{**args, **kw})
    pk.photon_qk_norm_rope_kv_cache_write_int8(None, None, k, v, pos, slots, None, w, 1e-6, pool, 1e4)
    torch.cuda.synchronize()
    assert pk.photon_device_errors() == 0
