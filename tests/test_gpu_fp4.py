"""4-bit (E2M1) KV cache on the GPU: write, read and decode against the
oracle's definitions (oracle/fp4.py), and the step a program makes of them."""
import numpy as np
import pytest

import oracle
import synth
from oracle import fp4
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu


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
    """Pool of random codes and bf16 scales of about std / 3."""
    byte, nib, sb = fp4.record_positions(d)
    pool = rng.integers(0, 256, (nb, H, 17 * d), dtype=np.uint8)
    sc = np.abs(rng.standard_normal((2, 16, d // 64) + (nb, H)) * std / 3 + std / 6).astype(np.float32)
    bits = (sc.view(np.uint32) >> 16).astype(np.uint16)
    for w in range(2):
        pool[:, :, sb[w]] = np.moveaxis(bits[w] & 0xFF, (0, 1), (2, 3)).astype(np.uint8)
        pool[:, :, sb[w] + 1] = np.moveaxis(bits[w] >> 8, (0, 1), (2, 3)).astype(np.uint8)
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


def _decode(pk, q, pool, bt, ctx, scale, out_dtype, part, max_ctx=None, extra_rows=0):
    torch = _torch()
    B, Hq, d = q.shape
    mc = int(max(max(ctx), 1)) if max_ctx is None else max_ctx
    n = pk.photon_paged_attention_workspace_size(B, Hq, d, mc, part)
    ws = torch.randint(0, 256, (max(n, 1),), dtype=torch.uint8, device="cuda") if n else None
    out = torch.full((B + extra_rows, Hq, d), -7.0, dtype=out_dtype, device="cuda")
    pk.photon_paged_attention_decode_fp4(q, pool, _dev(bt), _dev(np.asarray(ctx, np.int32)), scale, out[:B], mc, part, ws)
    torch.cuda.synchronize()
    return out


def _tolerance(q64, kd, vd, ctx, scale, out_bf16, ref):
    """Per output element.  Let V = max |v|.  A relative error e of a weight
    moves a weighted mean by at most 2 e V (numerator and denominator), one of
    the numerator's weights alone by e V.
      score: products of f16 by exact codes summed in fp32, at most d + 4
        roundings of 2^-24 (2^-23 where the tensor core truncates) of
        sum |q||k|, times the scale; ex2 within 2^-22
      weight times V scale in f16: 2^-12 (bf16 output) or f16 + remainder 2^-22
      sums over n tokens in fp32, one rounding per 16-token MMA: (n / 16 + 8) 2^-23
      output: half a step of the type, 2^-8 or 2^-24 of the value"""
    d = q64.shape[-1]
    V = np.abs(vd).max() if vd.size else 0.0
    qk = np.abs(q64).sum(-1).max() * np.abs(kd).max()
    e_score = abs(scale) * (d + 4) * 2.0 ** -23 * qk + 2.0 ** -22
    e_sum = (max(ctx) / 16 + 8) * 2.0 ** -23
    e_p = 2.0 ** -12 if out_bf16 else 2.0 ** -22
    return V * (2 * e_score + 2 * e_sum + e_p) + np.abs(ref) * (2.0 ** -8 if out_bf16 else 2.0 ** -24)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("style", ["neox", "gptj", "none"])
@pytest.mark.parametrize("T,H", [(1, 1), (5, 3), (37, 8), (70, 4)])
def test_write_codes_equal_the_oracle(T, H, style, dtype, d):
    """Every byte of the pool: codes and scales of the written tokens bit for
    bit, all other bytes as they were; slots -1 and past the pool write nothing."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(T * 10 + H + d)
    nb = 12
    k, kt = _storage(rng.standard_normal((T, H, d)) * 0.7, dtype)
    v, vt = _storage(rng.standard_normal((T, H, d)) * rng.lognormal(0, 3, (T, H, 1)), dtype)
    slots = rng.permutation(nb * 16)[:T].astype(np.int64)
    slots[T // 2::7] = -1
    pos = rng.integers(0, 100000, T).astype(np.int32)
    want = rng.integers(0, 256, (nb, H, 17 * d), dtype=np.uint8)
    pool = _dev(want.copy())
    gpu_slots = slots.copy()
    if T > 4:
        gpu_slots[slots < 0] = np.where(np.arange((slots < 0).sum()) % 2, nb * 16 + 3, -1)
    pk.photon_device_errors()
    pk.photon_kv_cache_write_fp4(kt, vt, _dev(pos), _dev(gpu_slots), pool, 5e5, style)
    fp4.write(k, v, pos, slots, want, 5e5, {"neox": 0, "gptj": 1, "none": 2}[style])
    assert np.array_equal(pool.cpu().numpy(), want)
    assert pk.photon_device_errors() == (pk.DEVERR_SLOT_RANGE if (gpu_slots >= nb * 16).any() else 0)


@pytest.mark.parametrize("T,H,d", [(5003, 1, 64), (1301, 2, 128), (700, 3, 64)])
def test_write_of_long_batches_equals_the_oracle(T, H, d):
    """Tiles of several tokens per CTA with a ragged end, skipped and
    out-of-pool slots among them; untouched bytes as they were."""
    pk = ensure_built()
    rng = np.random.default_rng(T)
    nb = T // 16 + 5
    k, kt = _storage(rng.standard_normal((T, H, d)), "bf16")
    v, vt = _storage(rng.standard_normal((T, H, d)) * 3, "bf16")
    slots = rng.permutation(nb * 16)[:T].astype(np.int64)
    slots[::17] = -1
    gpu_slots = slots.copy()
    gpu_slots[17] = nb * 16 + 5
    pos = rng.integers(0, 2 ** 20, T).astype(np.int32)
    want = rng.integers(0, 256, (nb, H, 17 * d), dtype=np.uint8)
    pool = _dev(want.copy())
    pk.photon_device_errors()
    pk.photon_kv_cache_write_fp4(kt, vt, _dev(pos), _dev(gpu_slots), pool, 1e6)
    fp4.write(k, v, pos, slots, want, 1e6)
    assert np.array_equal(pool.cpu().numpy(), want)
    assert pk.photon_device_errors() == pk.DEVERR_SLOT_RANGE


@pytest.mark.parametrize("style", ["neox", "gptj"])
def test_write_rotates_infinities_and_nans_into_nan_groups(style):
    """A pair that holds an infinity or a NaN makes the groups of both its
    dims NaN, at position 0 too; the row's other group is as without it."""
    pk = ensure_built()
    rng = np.random.default_rng(3)
    d, T = 128, 4
    x = rng.standard_normal((T, 1, d)).astype(np.float32)
    x[1, 0, 3], x[2, 0, 3], x[3, 0, 70] = np.inf, np.nan, -np.inf
    pos = np.array([5, 0, 1000, 17], np.int32)
    pool = _dev(np.zeros((1, 1, 17 * d), np.uint8))
    _, xt = _storage(x, "bf16")
    pk.photon_kv_cache_write_fp4(xt, xt, _dev(pos), _dev(np.arange(T, dtype=np.int64)), pool, 1e4, style)
    kd, vd = fp4.dequant(pool.cpu().numpy(), d)
    nan = np.isnan(kd[0, 0, :T]).reshape(T, 2, 64).all(-1)
    fine = np.isfinite(kd[0, 0, :T]).reshape(T, 2, 64).all(-1)
    both = style == "neox"                                  # dims 3 and 67 are a pair
    assert nan.tolist() == [[False, False], [True, both], [True, both], [both, True]]
    assert np.array_equal(fine, ~nan)
    assert np.isnan(vd[0, 0, :T]).reshape(T, 2, 64).all(-1).tolist() == [[False, False], [True, False],
                                                                       [True, False], [False, True]]


@pytest.mark.parametrize("d", [64, 128])
def test_write_midpoints_and_special_groups(d):
    """fp32 rows whose quotient by the group's scale is exactly a midpoint, or
    one unit beside it; groups of zeros, of subnormals, of huge values, with an
    infinity or a NaN."""
    pk = ensure_built()
    rng = np.random.default_rng(d)
    T, H, nb = 32, 2, 2
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x = np.zeros((T, H, d), np.float32)
    for t in range(T):
        for h in range(H):
            for g in range(d // 64):
                s = float(np.float32(rng.integers(128, 256)) * np.float32(2.0) ** int(rng.integers(-90, 100)))
                y = (mids[rng.integers(0, 7, 64)] * rng.choice([-1, 1], 64) * s).astype(np.float32)
                nudge = rng.integers(0, 3, 64)
                y = np.where(nudge == 1, np.nextafter(y, np.float32(np.inf)),
                             np.where(nudge == 2, np.nextafter(y, np.float32(-np.inf)), y))
                y[rng.integers(0, 64)] = np.float32(6 * s)
                x[t, h, 64 * g:64 * g + 64] = y
    x[0] = 0
    x[1] = rng.standard_normal((H, d)).astype(np.float32) * np.float32(2.0 ** -132)
    x[2, 0, 5], x[3, 1, 7], x[4, 0, 9] = np.inf, np.nan, -np.inf
    x[5] = np.float32(3.0e38) * rng.choice([-1, 1, 0.5], (H, d))
    slots = rng.permutation(nb * 16).astype(np.int64)
    pos = np.zeros(T, np.int32)
    want = np.zeros((nb, H, 17 * d), np.uint8)
    pool = _dev(want.copy())
    pk.photon_kv_cache_write_fp4(_dev(x), _dev(-x), _dev(pos), _dev(slots), pool, 1e4, "none")
    fp4.write(x, -x, pos, slots, want, 1e4, oracle.ROPE_NONE)
    kd, vd = fp4.dequant(want, d)
    kg, vg = fp4.dequant(pool.cpu().numpy(), d)
    assert np.array_equal(kg, kd, equal_nan=True) and np.array_equal(vg, vd, equal_nan=True)
    blk, off = slots // 16, slots % 16
    assert np.isnan(kg[blk[2], 0, off[2], :64]).all() and np.isnan(vg[blk[3], 1, off[3], :64]).all()
    assert np.isfinite(kg[blk[5], :, off[5]]).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(1, 1), (33, 3), (200, 8)])
def test_read_returns_the_rounded_values(T, H, dtype, d):
    """Bit for bit the product rounded once; repeated slots; rows of slots -1
    or past the pool left as they were."""
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
    k = torch.full((T, H, d), -3.0, dtype=dt, device="cuda")
    v = torch.full((T, H, d), -3.0, dtype=dt, device="cuda")
    pk.photon_device_errors()
    pk.photon_kv_cache_read_fp4(_dev(pool), _dev(slots), k, v)
    torch.cuda.synchronize()
    for got, val in zip((k, v), fp4.dequant(pool, d)):
        want = val[np.clip(slots, 0, nb * 16 - 1) // 16, :, np.clip(slots, 0, nb * 16 - 1) % 16]
        want = torch.from_numpy(np.where(skip[:, None, None], -3.0, want)).float().to(dt)
        assert torch.equal(got.cpu(), want)
    assert pk.photon_device_errors() == (pk.DEVERR_SLOT_RANGE if (slots >= nb * 16).any() else 0)


def test_read_longer_than_one_grid():
    """More tokens than one launch's tiles: every row, at its own place."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(9)
    d, nb, T = 64, 3, 64 * 65535 + 77
    pool = _random_pool(rng, nb, 1, d)
    slots = torch.randint(0, nb * 16, (T,), generator=torch.Generator().manual_seed(1)).cuda()
    k, v = (torch.empty(T, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pk.photon_kv_cache_read_fp4(_dev(pool), slots, k, v)
    for got, val in zip((k, v), fp4.dequant(pool, d)):
        rows = torch.from_numpy(val[:, 0].reshape(nb * 16, d)).float().bfloat16().cuda()
        assert torch.equal(got[:, 0], rows[slots])


CONTEXTS = [([1, 17, 600, 1500, 33, 0], 256), ([3000, 9, 700, 0, 16], 512),
            ([16, 31, 32, 33, 47, 48, 49, 63, 64, 65, 511, 512, 513, 15], 64), ([1024], 32), ([5], 512), ([130, 0], 16)]


@pytest.mark.parametrize("ctx,part", CONTEXTS)
@pytest.mark.parametrize("H,G", [(8, 1), (8, 2), (8, 4), (4, 8), (1, 4), (3, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_decode_matches_the_oracle(ctx, part, H, G, d, out):
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(sum(ctx) + H * G + d)
    nb = sum(-(-c // 16) for c in ctx) + 3
    pool = _random_pool(rng, nb, H, d)
    bt = _tables(rng, ctx, nb)
    q, qt = _storage(rng.standard_normal((len(ctx), H * G, d)), "bf16")
    scale = d ** -0.5
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    got = _decode(pk, qt, _dev(pool), bt, ctx, scale, dt, part, extra_rows=2)
    ref = fp4.paged_attention(q, pool, bt, ctx, scale)
    assert (got[len(ctx):] == -7.0).all()                  # rows behind the batch
    got = got[:len(ctx)].double().cpu().numpy()
    kd, vd = fp4.dequant(pool, d)
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= _tolerance(oracle.to_f64(q), kd, vd, ctx, scale, out == "bf16", ref)).all()
    for s, c in enumerate(ctx):
        if c == 0:
            assert (got[s] == 0).all()
    assert pk.photon_device_errors() == 0


@pytest.mark.parametrize("qexp,vexp,scale", [(0, 0, -0.3), (100, 0, 2.0 ** -103), (-100, 0, 2.0 ** 97), (126, 0, 0.0), (123, 0, 2.0 ** -126), (120, 0, 0.0),
                                             (0, 60, 0.125), (0, -100, 0.125), (3, -60, -0.01), (-130, 0, 0.5)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_is_scale_free(qexp, vexp, scale, d):
    """q and V scales of any magnitude, a negative or zero softmax scale."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(7)
    ctx, H, G = [300, 40, 1], 2, 4
    nb = 30
    pool = _random_pool(rng, nb, H, d)
    byte, nib, sb = fp4.record_positions(d)
    lo, hi = pool[:, :, sb[1]].astype(np.uint16), pool[:, :, sb[1] + 1].astype(np.uint16)
    bits = (lo | (hi << 8)).astype(np.int64) + (vexp << 7)
    bits = np.where(rng.random(bits.shape) < 0.2, 0, bits).astype(np.uint16)     # groups of zeros
    pool[:, :, sb[1]], pool[:, :, sb[1] + 1] = bits & 0xFF, bits >> 8
    bt = _tables(rng, ctx, nb)
    q, qt = _storage(rng.standard_normal((3, H * G, d)) * 2.0 ** qexp, "bf16")
    got = _decode(pk, qt, _dev(pool), bt, ctx, scale, torch.float32, 64).double().cpu().numpy()
    ref = fp4.paged_attention(q, pool, bt, ctx, float(np.float32(scale)))
    kd, vd = fp4.dequant(pool, d)
    # 2^126 times a normal value of 4 or more is an infinity in bf16: rows whose q holds one are NaN in the
    # definition too (infinity times the zero scale)
    fine = np.isfinite(ref)
    assert np.array_equal(np.isfinite(got), fine) and (fine.all() or qexp == 126)
    q64 = np.where(np.isfinite(oracle.to_f64(q)), oracle.to_f64(q), 0.0)
    off = np.abs(got - ref)[fine]
    assert (off <= (_tolerance(q64, kd, vd, ctx, scale, False, ref) + 2.0 ** -149)[fine]).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("part", [32, 512])
def test_decode_ignores_everything_past_the_context(d, part):
    """NaN and infinite scales behind the last token, in the page's tail and in
    unused blocks, leave every bit of the output as it was."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(d + part)
    ctx, H, G = [1, 15, 37, 200, 449, 64], 2, 4
    nb = 80
    pool = _random_pool(rng, nb, H, d)
    bt = _tables(rng, ctx, nb, width=32)
    _, qt = _storage(rng.standard_normal((len(ctx), H * G, d)), "bf16")
    a = _decode(pk, qt, _dev(pool), bt, ctx, 0.2, torch.float32, part)
    byte, nib, sb = fp4.record_positions(d)
    bad = np.ones((nb, 16), bool)
    for s, c in enumerate(ctx):
        for p in range(c):
            bad[bt[s, p // 16], p % 16] = False
    for b, r in zip(*np.nonzero(bad)):
        for w in range(2):
            pool[b][:, sb[w, r]] = 0xC0 if (b + r) % 2 else 0x80
            pool[b][:, sb[w, r] + 1] = 0x7F                     # NaN, +inf
            pool[b][:, byte[w, r]] = 0xFF
    b_ = _decode(pk, qt, _dev(pool), bt, ctx, 0.2, torch.float32, part)
    assert torch.equal(a, b_) and torch.isfinite(a).all()
    assert pk.photon_device_errors() == 0


def test_decode_nan_values_stay_in_their_heads_and_rows():
    """A token with a NaN V scale makes the outputs of its (sequence, KV head)
    NaN in the dims of that scale, one with a NaN K scale in all; no others."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(5)
    d, ctx, H, G, nb = 128, [100, 300, 50], 2, 2, 40
    pool = _random_pool(rng, nb, H, d)
    bt = _tables(rng, ctx, nb)
    byte, nib, sb = fp4.record_positions(d)
    pool[bt[0, 2], 1, sb[1, 3, 1]:sb[1, 3, 1] + 2] = [0xFF, 0x7F]
    pool[bt[1, 4], 0, sb[0, 8, 0]:sb[0, 8, 0] + 2] = [0xFF, 0x7F]
    _, qt = _storage(rng.standard_normal((3, H * G, d)), "bf16")
    for part in (64, 512):
        got = torch.isnan(_decode(pk, qt, _dev(pool), bt, ctx, 0.1, torch.float32, part)).cpu().numpy()
        want = np.zeros_like(got)
        want[0, 2:4, 64:] = True
        want[1, 0:2] = True
        assert np.array_equal(got, want)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_bad_blocks_and_contexts(d):
    """Block ids outside the pool are skipped and flagged, a context above the
    declared bound is clamped and flagged; the rest is as without them."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(d)
    ctx, H, G, nb = [100, 200, 33, 64], 2, 4, 40
    pool = _random_pool(rng, nb, H, d)
    bt = _tables(rng, ctx, nb)
    q, qt = _storage(rng.standard_normal((4, H * G, d)), "bf16")
    bad = bt.copy()
    bad[0, 1], bad[1, 3], bad[1, 12] = nb, -5, 2 ** 30
    bad[2, :3] = -1                                     # nothing left of sequence 2
    pk.photon_device_errors()
    for part in (32, 512):
        got = _decode(pk, qt, _dev(pool), bad, ctx, 0.2, torch.float32, part).double().cpu().numpy()
        assert pk.photon_device_errors() == pk.DEVERR_BLOCK_RANGE
        kd, vd = fp4.dequant(pool, d)
        q64 = oracle.to_f64(q)
        for s, c in enumerate(ctx):
            keep = np.array([0 <= bad[s, p // 16] < nb for p in range(c)])
            for h in range(H * G):
                if not keep.any():
                    assert (got[s, h] == 0).all()
                    continue
                ks = np.array([kd[bad[s, p // 16], h // G, p % 16] for p in range(c) if keep[p]])
                vs = np.array([vd[bad[s, p // 16], h // G, p % 16] for p in range(c) if keep[p]])
                x = ks @ q64[s, h] * 0.2
                w = np.exp(x - x.max())
                ref = w @ vs / w.sum()
                assert (np.abs(got[s, h] - ref) <= _tolerance(q64, kd, vd, ctx, 0.2, False, ref)).all()
    long = [100, 10 ** 6, 33, 64]
    got = _decode(pk, qt, _dev(pool), bt, long, 0.2, torch.float32, 64, max_ctx=208)
    assert pk.photon_device_errors() & pk.DEVERR_CONTEXT_RANGE
    same = _decode(pk, qt, _dev(pool), bt, [100, 208, 33, 64], 0.2, torch.float32, 64, max_ctx=208)
    assert torch.equal(got, same)
    pk.photon_device_errors()


@pytest.mark.parametrize("H,G,d", [(8, 4, 64), (1, 8, 64), (3, 2, 128), (8, 2, 128)])
@pytest.mark.parametrize("kind", ["long", "ragged", "mostly empty"])
def test_decode_of_full_grids(H, G, d, kind):
    """Batches that give every warp of the grid several pages and partitions,
    with empty and one-token sequences, hundreds in a row among them; every
    call gives the same bits."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(H * 7 + d)
    total = 16 * 5 * (2432 // H)
    if kind == "long":
        ctx = [int(x) for x in rng.integers(total // 8, total // 3, 8)]
    elif kind == "ragged":
        ctx = [int(x) for x in np.clip(rng.lognormal(5.5, 1.2, 2 * total // 500), 1, 6000)]
    else:
        ctx = [0] * 300 + [int(x) for x in rng.integers(1, 40, 50)] + [0] * 500 + [total] + [0, 1, 0, 16] + [0] * 200
    nb = sum(-(-c // 16) for c in ctx) + 1
    pool = _random_pool(rng, nb, H, d)
    bt = _tables(rng, ctx, nb)
    q, qt = _storage(rng.standard_normal((len(ctx), H * G, d)), "bf16")
    dev = _dev(pool)
    a = _decode(pk, qt, dev, bt, ctx, d ** -0.5, torch.float32, 16)
    for _ in range(4):
        assert torch.equal(a, _decode(pk, qt, dev, bt, ctx, d ** -0.5, torch.float32, 16))
    ref = fp4.paged_attention(q, pool, bt, ctx, d ** -0.5)
    kd, vd = fp4.dequant(pool, d)
    tol = _tolerance(oracle.to_f64(q), kd, vd, ctx, d ** -0.5, False, ref)
    assert (np.abs(a.double().cpu().numpy() - ref) <= tol).all()
    assert pk.photon_device_errors() == 0


@pytest.mark.parametrize("G,d,H", [(4, 64, 8), (1, 64, 8), (2, 128, 8), (8, 128, 16)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_decode_declared_long(G, d, H, out):
    """A batch whose declared bound asks for the long steps' kernel (192 pages
    per warp and more), the contexts themselves short, ragged, empty or long;
    garbage behind each, and a bad block id."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(G + d)
    ctx = [3001, 0, 1, 129, 128, 127, 16, 700]
    width = -(-192 * 16 * 160 // (len(ctx) * H)) + 1
    nb = sum(-(-c // 16) for c in ctx) + 2
    pool = _random_pool(rng, nb, H, d)
    bt = _tables(rng, ctx, nb, width=width)
    bt[:, 200:] = 7                                       # past every context: never read
    q, qt = _storage(rng.standard_normal((len(ctx), H * G, d)), "bf16")
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    clean = pool.copy()
    byte, nib, sb = fp4.record_positions(d)
    for s, c in enumerate(ctx):
        for r in range(c % 16, 16 if c % 16 else 0):
            for w in range(2):
                pool[bt[s, c // 16]][:, sb[w, r]] = 0x80
                pool[bt[s, c // 16]][:, sb[w, r] + 1] = 0x7F
    pk.photon_device_errors()
    got = _decode(pk, qt, _dev(pool), bt, ctx, d ** -0.5, dt, 64, max_ctx=width * 16)
    assert torch.equal(got, _decode(pk, qt, _dev(pool), bt, ctx, d ** -0.5, dt, 64, max_ctx=width * 16))
    ref = fp4.paged_attention(q, clean, bt, ctx, d ** -0.5)
    kd, vd = fp4.dequant(clean, d)
    tol = _tolerance(oracle.to_f64(q), kd, vd, ctx, d ** -0.5, out == "bf16", ref)
    assert (np.abs(got.double().cpu().numpy() - ref) <= tol).all()
    assert pk.photon_device_errors() == 0
    bt[3, 2] = -3
    again = _decode(pk, qt, _dev(pool), bt, ctx, d ** -0.5, dt, 64, max_ctx=width * 16)
    rows = [s for s in range(len(ctx)) if s != 3]
    assert torch.equal(again[rows], got[rows]) and torch.isfinite(again).all()
    assert pk.photon_device_errors() == pk.DEVERR_BLOCK_RANGE


def test_decode_on_another_stream_and_two_at_once():
    """Two decodes on two streams, each with its own workspace: the results of
    one after the other."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(4)
    ctx = [int(x) for x in rng.integers(1, 3000, 24)]
    nb = sum(-(-c // 16) for c in ctx)
    pool, bt = _dev(_random_pool(rng, nb, 4, 64)), _dev(_tables(rng, ctx, nb))
    cl = _dev(np.array(ctx, np.int32))
    _, qa = _storage(rng.standard_normal((24, 16, 64)), "bf16")
    _, qb = _storage(rng.standard_normal((24, 16, 64)), "bf16")
    n = pk.photon_paged_attention_workspace_size(24, 16, 64, max(ctx), 64)
    ws = [torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty(24, 16, 64, device="cuda") for _ in range(4)]
    args = lambda q, i: (q, pool, bt, cl, 0.125, outs[i], max(ctx), 64, ws[i & 1])
    pk.photon_paged_attention_decode_fp4(*args(qa, 0))
    pk.photon_paged_attention_decode_fp4(*args(qb, 1))
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        pk.photon_paged_attention_decode_fp4(*args(qa, 2), stream=sa)
        with torch.cuda.stream(sb):
            pk.photon_paged_attention_decode_fp4(*args(qb, 3))
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])


def test_many_kv_heads():
    """As many KV heads as a call takes: write, read and decode."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(12)
    H, d, ctx = 1024, 64, [40, 17]
    pool = _random_pool(rng, 6, H, d)
    bt = _tables(rng, ctx, 6)
    q, qt = _storage(rng.standard_normal((2, H, d)), "bf16")
    for part in (16, 512):
        got = _decode(pk, qt, _dev(pool), bt, ctx, 0.1, torch.float32, part).double().cpu().numpy()
        ref = fp4.paged_attention(q, pool, bt, ctx, 0.1)
        kd, vd = fp4.dequant(pool, d)
        assert (np.abs(got - ref) <= _tolerance(oracle.to_f64(q), kd, vd, ctx, 0.1, False, ref)).all()
    k, kt = _storage(rng.standard_normal((2, H, d)), "bf16")
    dev, slots = _dev(pool.copy()), np.array([5, 90], np.int64)
    pk.photon_kv_cache_write_fp4(kt, kt, _dev(np.array([3, 4], np.int32)), _dev(slots), dev, 1e4)
    fp4.write(k, k, [3, 4], slots, pool, 1e4)
    assert np.array_equal(dev.cpu().numpy(), pool)
    ko, vo = torch.empty_like(kt), torch.empty_like(kt)
    pk.photon_kv_cache_read_fp4(dev, _dev(slots), ko, vo)
    want = fp4.dequant(pool, d)[1][slots // 16, :, slots % 16]
    assert torch.equal(vo.cpu(), torch.from_numpy(want).float().bfloat16())


@pytest.mark.parametrize("ctx,part", [
    ([500, 1, 0, 128, 129, 33, 16, 512], 512),                                   # one piece per row, no workspace
    ([0, 0, 1, 15, 16, 17, 32, 0, 130, 1000, 47, 0, 1, 1, 1, 1, 1, 64, 5, 0], 128),  # runs over many sequences
    ([16 * k + k % 3 for k in range(1, 36)], 256),                               # every share of 1 to 16 pages
    ([3001], 512), ([700, 4090], 1024),
    ([500 - 3 * k for k in range(160)], 512),                                    # two items to some CTAs
    ([(97 * k) % 1200 for k in range(90)], 256)])                                # runs over pieces of 16 pages, many
@pytest.mark.parametrize("H,G,d", [(2, 4, 64), (1, 8, 128), (3, 1, 128), (4, 2, 64)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_decode_of_few_long_pieces(ctx, part, H, G, d, out):
    """Batches far smaller than the GPU with large partitions: the warps of a
    CTA share each piece.  Missing blocks empty some of the shares; every call
    gives the same bits."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(len(ctx) + part + d)
    nb = sum(-(-c // 16) for c in ctx) + 1
    pool = _random_pool(rng, nb, H, d)
    bt = _tables(rng, ctx, nb)
    q, qt = _storage(rng.standard_normal((len(ctx), H * G, d)), "bf16")
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    dev = _dev(pool)
    pk.photon_device_errors()
    a = _decode(pk, qt, dev, bt, ctx, d ** -0.5, dt, part, extra_rows=1)
    assert torch.equal(a, _decode(pk, qt, dev, bt, ctx, d ** -0.5, dt, part, extra_rows=1))
    assert (a[len(ctx):] == -7.0).all()
    ref = fp4.paged_attention(q, pool, bt, ctx, d ** -0.5)
    kd, vd = fp4.dequant(pool, d)
    q64 = oracle.to_f64(q)
    tol = _tolerance(q64, kd, vd, ctx, d ** -0.5, out == "bf16", ref)
    assert (np.abs(a[:len(ctx)].double().cpu().numpy() - ref) <= tol).all()
    assert pk.photon_device_errors() == 0
    # a sequence's first pages alone, then its last one alone, are left
    s = int(np.argmax(ctx))
    n = -(-ctx[s] // 16)
    for keep in (range(0, 2), range(n - 1, n)):
        some = bt.copy()
        some[s, [i for i in range(n) if i not in keep]] = -1
        got = _decode(pk, qt, dev, some, ctx, d ** -0.5, dt, part)
        assert pk.photon_device_errors() == pk.DEVERR_BLOCK_RANGE
        rest = [i for i in range(len(ctx)) if i != s]
        assert torch.equal(got[rest], a[rest])
        tokens = [p for p in range(ctx[s]) if p // 16 in keep]
        for h in range(H * G):
            ks = np.array([kd[bt[s, p // 16], h // G, p % 16] for p in tokens])
            vs = np.array([vd[bt[s, p // 16], h // G, p % 16] for p in tokens])
            x = ks @ q64[s, h] * d ** -0.5
            w = np.exp(x - x.max())
            want = w @ vs / w.sum()
            lim = _tolerance(q64, kd, vd, ctx, d ** -0.5, out == "bf16", want)
            assert (np.abs(got[s, h].double().cpu().numpy() - want) <= lim).all()


def test_decode_repeats_bit_for_bit():
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(1)
    ctx = [int(x) for x in rng.integers(1, 4000, 40)]
    nb = sum(-(-c // 16) for c in ctx)
    pool = _dev(_random_pool(rng, nb, 4, 64))
    bt = _tables(rng, ctx, nb)
    _, qt = _storage(rng.standard_normal((40, 16, 64)), "bf16")
    a = _decode(pk, qt, pool, bt, ctx, 0.125, torch.float32, 128)
    for _ in range(5):
        assert torch.equal(a, _decode(pk, qt, pool, bt, ctx, 0.125, torch.float32, 128))


def test_large_pool_offsets():
    """Records past 2^32 bytes: written, read back and attended to."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(2)
    d, H = 128, 8
    nb = 2 ** 32 // (17 * d * H) + 40
    pool = torch.zeros(nb, H, 17 * d, dtype=torch.uint8, device="cuda")
    ctx = [50]
    bt = np.array([[nb - 1, 3, nb - 7, nb - 2]], np.int32)
    pos = np.arange(50, dtype=np.int32)
    slots = bt[0, pos // 16].astype(np.int64) * 16 + pos % 16
    k, kt = _storage(rng.standard_normal((50, H, d)), "bf16")
    v, vt = _storage(rng.standard_normal((50, H, d)), "bf16")
    pk.photon_kv_cache_write_fp4(kt, vt, _dev(pos), _dev(slots), pool, 1e4)
    small = np.zeros((4, H, 17 * d), np.uint8)
    fp4.write(k, v, pos, np.arange(50, dtype=np.int64), small, 1e4)
    assert np.array_equal(pool[bt[0].tolist()].cpu().numpy(), small)
    ko, vo = torch.empty_like(kt, dtype=torch.float32), torch.empty_like(vt, dtype=torch.float32)
    pk.photon_kv_cache_read_fp4(pool, _dev(slots), ko, vo)
    kd, vd = fp4.dequant(small, d)
    assert np.array_equal(ko.cpu().numpy(), kd[pos // 16, :, pos % 16].astype(np.float32))
    q, qt = _storage(rng.standard_normal((1, 16, d)), "bf16")
    got = _decode(pk, qt, pool, bt, ctx, 0.1, torch.float32, 512).double().cpu().numpy()
    ref = fp4.paged_attention(q, small, np.arange(4, dtype=np.int32)[None], ctx, 0.1)
    assert (np.abs(got - ref) <= _tolerance(oracle.to_f64(q), kd, vd, ctx, 0.1, False, ref)).all()
    assert pk.photon_device_errors() == 0


def _raise_v_scales(pool, bt, s, tokens, exps, plane=None):
    """Multiplies the V scales of `tokens` of sequence s by 2^exps (None: makes
    them 0), in every plane or in one; in place."""
    byte, nib, sb = fp4.record_positions(pool.shape[-1] // 17)
    for p, e in zip(tokens, exps):
        rec = pool[bt[s, p // 16]]
        at = sb[1, p % 16] if plane is None else sb[1, p % 16, plane:plane + 1]
        bits = rec[:, at].astype(np.int64) | (rec[:, at + 1].astype(np.int64) << 8)
        bits = np.zeros_like(bits) if e is None else bits + (e << 7)
        rec[:, at], rec[:, at + 1] = bits & 0xFF, bits >> 8


# one warp's steps in turn; a team's shares; split pieces; teams of pieces; long steps
GROWING = [([48, 33, 35], 512, None), ([64, 500, 130], 512, None), ([300, 200, 90], 32, None),
           ([3000, 700, 1500], 512, None), ([700, 33, 90, 1500], 64, 192 * 16 * 160)]


@pytest.mark.parametrize("ctx,part,bound", GROWING)
@pytest.mark.parametrize("early,late", [(None, 40), (None, 110), (-100, 40), (0, 60), (40, None), (110, -100)])
@pytest.mark.parametrize("H,G,d", [(2, 4, 64), (2, 2, 128)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_decode_of_values_that_grow_or_vanish(ctx, part, bound, early, late, H, G, d, out):
    """Values of one magnitude in a context's first tokens and of another in
    the rest: no magnitude of a value changes how much a token's score counts."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(sum(ctx) + d)
    mc = max(ctx) if bound is None else -(-bound // (len(ctx) * H) // 16) * 16
    nb = sum(-(-c // 16) for c in ctx) + 1
    pool = _random_pool(rng, nb, H, d)
    bt = _tables(rng, ctx, nb, width=-(-mc // 16))
    for s, c in enumerate(ctx):
        cut = min(32, c - 1) if c < 64 else c // 2
        _raise_v_scales(pool, bt, s, range(c), [early if p < cut else late for p in range(c)])
    q, qt = _storage(rng.standard_normal((len(ctx), H * G, d)) * 0.1, "bf16")
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    got = _decode(pk, qt, _dev(pool), bt, ctx, d ** -0.5, dt, part, max_ctx=mc).double().cpu().numpy()
    kd, vd = fp4.dequant(pool, d)
    for s, c in enumerate(ctx):
        one = fp4.paged_attention(q[s:s + 1], pool, bt[s:s + 1], [c], d ** -0.5)
        mine = vd[bt[s, :-(-c // 16)]].transpose(0, 2, 1, 3).reshape(-1, H, d)[:c]
        tol = _tolerance(oracle.to_f64(q), kd, mine, [c], d ** -0.5, out == "bf16", one)
        assert (np.abs(got[s:s + 1] - one) <= tol).all()
    assert pk.photon_device_errors() == 0


@pytest.mark.parametrize("part", [32, 512])
@pytest.mark.parametrize("exp", [40, -60, 100])
def test_decode_planes_of_different_magnitude(part, exp):
    """Each 64 dims have scales of their own: large ones in one plane leave the
    other plane's outputs as exact as they were."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(part)
    ctx, H, G, d, nb = [300, 40, 1, 700], 2, 4, 128, 70
    pool = _random_pool(rng, nb, H, d)
    bt = _tables(rng, ctx, nb)
    for s, c in enumerate(ctx):
        _raise_v_scales(pool, bt, s, range(c), [exp] * c, plane=0)
    q, qt = _storage(rng.standard_normal((4, H * G, d)), "bf16")
    for dt in (torch.bfloat16, torch.float32):
        got = _decode(pk, qt, _dev(pool), bt, ctx, 0.1, dt, part).double().cpu().numpy()
        ref = fp4.paged_attention(q, pool, bt, ctx, 0.1)
        kd, vd = fp4.dequant(pool, d)
        live = np.zeros((nb, 16), bool)
        for s, c in enumerate(ctx):
            for p in range(c):
                live[bt[s, p // 16], p % 16] = True
        for x in (slice(0, 64), slice(64, 128)):
            vx = np.where(live[:, None, :, None], vd, 0.0)[..., x]
            tol = _tolerance(oracle.to_f64(q), kd, vx, ctx, 0.1, dt is torch.bfloat16, ref[..., x])
            assert (np.abs(got[..., x] - ref[..., x]) <= tol).all()


@pytest.mark.parametrize("kexp", [116, 60, -60, -110])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("part", [32, 512])
def test_decode_keys_of_any_magnitude(kexp, d, part):
    """Keys up to just below 2^119 and down to 2^-112, the softmax scale
    bringing their scores back to a few units."""
    torch = _torch()
    pk = ensure_built()
    rng = np.random.default_rng(kexp + 200)
    ctx, H, G, nb = [300, 40, 1], 2, 4, 30
    pool = _random_pool(rng, nb, H, d)
    byte, nib, sb = fp4.record_positions(d)
    bits = (pool[:, :, sb[0]].astype(np.int64) | (pool[:, :, sb[0] + 1].astype(np.int64) << 8)) + (kexp << 7)
    pool[:, :, sb[0]], pool[:, :, sb[0] + 1] = bits & 0xFF, bits >> 8
    bt = _tables(rng, ctx, nb)
    q, qt = _storage(rng.standard_normal((3, H * G, d)), "bf16")
    kd, vd = fp4.dequant(pool, d)
    assert np.abs(kd).max() < 2.0 ** 119
    scale = float(np.float32(d ** -0.5 * 2.0 ** -kexp))
    got = _decode(pk, qt, _dev(pool), bt, ctx, scale, torch.float32, part).double().cpu().numpy()
    ref = fp4.paged_attention(q, pool, bt, ctx, scale)
    assert (np.abs(got - ref) <= _tolerance(oracle.to_f64(q), kd, vd, ctx, scale, False, ref)).all()
    assert pk.photon_device_errors() == 0
