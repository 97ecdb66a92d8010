"""8-bit KV cache with a scale per block and head, and the q/k norms: definitions
for the oracle in numpy, fp64, no code of the CUDA path.  Record layout: per
(block, KV head) 32 * d + 16 bytes for 16 tokens (see record_positions)."""
from __future__ import annotations

import numpy as np

import oracle

LEAST = np.float32(2.0 ** -100)   # smaller scales count as zero


def norm_rope(x, weight, eps, positions, rope_theta, rope_style=oracle.ROPE_NEOX):
    """fp64 rows [T, H, d]: RMS norm with weights [d] (None: none), then RoPE."""
    y = oracle.to_f64(x)
    if weight is not None:
        y = y * oracle.to_f64(weight) / np.sqrt((y * y).mean(-1, keepdims=True) + float(np.float32(eps)))
    if rope_style == oracle.ROPE_NONE or not y.size:
        return y
    return np.array([[oracle.rope(y[t, h], int(positions[t]), rope_theta, rope_style) for h in range(y.shape[1])]
                     for t in range(y.shape[0])]).reshape(y.shape)


def pair_length(y, rope_style):
    """Length of the rotation pair that each element of y [..., d] belongs to."""
    d = y.shape[-1]
    if rope_style == oracle.ROPE_GPTJ:
        return np.repeat(np.hypot(y[..., 0::2], y[..., 1::2]), 2, axis=-1)
    n = np.hypot(y[..., :d // 2], y[..., d // 2:])
    return np.concatenate([n, n], axis=-1)


def record_positions(d: int):
    """Byte of every code [2][16][d] of K (0) and V (1)."""
    byte = np.zeros((2, 16, d), np.int64)
    for r in range(16):
        a, rest = divmod(r, 4)
        n, j = divmod(rest, 2)
        for e in range(d):
            plane, x = divmod(e, 64)
            byte[0, r, e] = 1024 * plane + 64 * (8 * n + 2 * a + j) + x
            byte[1, r, e] = 16 * d + 1024 * plane + 512 * n + 16 * (4 * (x // 8) + a) + 8 * j + x % 8
    return byte


def scales(pool):
    """fp32 K and V scales [..., 2] of records [..., 32 d + 16]."""
    raw = np.ascontiguousarray(pool[..., -16:-8])
    return raw.view(np.float32)


def codes(pool, d):
    """Codes [nb, H, 16, d] (int) of K and V."""
    byte = record_positions(d)
    return [pool[:, :, byte[w]].astype(np.int64) - 128 for w in range(2)]


def dequant(pool, d):
    """fp64 K and V [nb, H, 16, d] of an 8-bit pool."""
    sc = scales(pool).astype(np.float64)
    return [c * sc[..., w][..., None, None] for w, c in enumerate(codes(pool, d))]


def new_scale(top, old):
    """The scale after a write whose largest magnitude is `top` (fp64 arrays)."""
    with np.errstate(all="ignore"):
        want = (np.asarray(top).astype(np.float32) / np.float32(127)).astype(np.float32)
        want = np.where(want < LEAST, np.float32(0), want)
        old = np.asarray(old, np.float32)
        grown = np.where(want > old, np.maximum(want, np.float32(2) * old), old).astype(np.float32)
    return np.where(np.isfinite(top), grown, np.float32(np.nan)).astype(np.float32)


def round_codes(x, factor):
    """x * factor (exact products in fp64) to the nearest integer, halves to even."""
    return np.rint(np.asarray(x, np.float64) * np.float64(factor)).astype(np.int64)


def write_rows(y, slots, pool, which, d, given=None):
    """In-place write of fp64 rows y [T, H, d] as K (0) or V (1).  given: an fp32
    array [nb, H] of scales to use in place of new_scale's where a block is
    written (a scale computed elsewhere, whose codes are to be checked)."""
    byte = record_positions(d)[which]
    T, H = y.shape[:2]
    runs, t = [], 0
    while t < T:
        n = 1
        if slots[t] >= 0:
            while t + n < T and n < 16 and slots[t + n] >= 0 and slots[t + n] // 16 == slots[t] // 16:
                n += 1
            runs.append((int(slots[t]) // 16, {int(slots[i]) % 16: i for i in range(t, t + n)}))
        t += n
    for b, rows in runs:
        for h in range(H):
            rec = pool[b, h]
            sc = rec[32 * d + 4 * which:32 * d + 4 * which + 4]
            old = sc.view(np.float32)[0]
            if 0 in rows:
                old = np.float32(0)
                rec[byte] = 128
            top = np.abs(y[list(rows.values()), h]).max()
            new = new_scale(top, old) if given is None else given[b, h]
            with np.errstate(all="ignore"):
                inv = np.float32(1) / new if new > 0 else np.float32(0)
                ratio = np.float32(old) * np.float32(inv)
            kept = [r for r in range(16) if r not in rows]
            if new > old and old > 0:
                rec[byte[kept]] = round_codes(rec[byte[kept]].astype(np.int64) - 128, ratio) + 128
            for r, i in rows.items():
                rec[byte[r]] = round_codes(y[i, h], inv) + 128 if new > 0 else 128
            sc[:] = np.array([new], np.float32).view(np.uint8)


def paged_attention(q, pool, block_tables, context_lens, scale):
    """Decode attention over the exactly dequantised values, fp64 [B, H_q, d]."""
    kd, vd = (np.ascontiguousarray(x) for x in dequant(pool, q.shape[-1]))
    return oracle.paged_attention(np.ascontiguousarray(oracle.to_f64(q)), kd, vd, block_tables, context_lens, scale)
