"""4-bit (E2M1) KV cache definitions for the oracle: numpy, fp64, no code of
the CUDA path.  Record layout: per (block, KV head) 17 * d bytes for 16 tokens
(see record_positions)."""
from __future__ import annotations

import numpy as np

import oracle

GROUP = 64


def decode(code: int) -> float:
    """Value of an E2M1 code: sign, exponent (bias 1), one mantissa bit."""
    e, m = (code >> 1) & 3, code & 1
    mag = m * 0.5 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)
    return -mag if code & 8 else mag


VALUES = np.array([decode(c) for c in range(16)])


def encode(y: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """Nearest code of y / scale (fp64 arrays, scale > 0), ties to the even
    code, saturating: by the distance |y| - value * scale to every code (the
    products and differences of bf16/fp32 operands are exact in fp64)."""
    dist = np.abs(np.abs(y)[..., None] - VALUES[:8] * scale[..., None])
    best = dist.min(-1, keepdims=True)
    tied = dist == best
    pick = np.where(tied[..., 0::2].any(-1), 2 * tied[..., 0::2].argmax(-1), 2 * tied[..., 1::2].argmax(-1) + 1)
    return (pick + np.where(y < 0, 8, 0)).astype(np.uint8)


def quantise(y: np.ndarray):
    """Codes [..., d] and bf16 scale bits [..., d / 64] of storage rows y
    (float32, or uint16 bf16 bits)."""
    f = oracle.to_f64(y)
    g = f.reshape(*f.shape[:-1], -1, GROUP)
    top = np.abs(g).max(-1)                     # NaN stays NaN
    with np.errstate(all="ignore"):
        quo = (top.astype(np.float32) / np.float32(6)).astype(np.float64)
    bits = np.array([oracle.round_bf16(q) if np.isfinite(t) else 0x7FFF
                     for q, t in zip(quo.ravel(), top.ravel())], np.uint16).reshape(top.shape)
    sc = oracle.bf16_to_f64(bits)[..., None]
    ok = np.isfinite(sc) & (sc > 0)
    codes = np.where(ok, encode(np.where(ok, g, 0.0), np.broadcast_to(np.where(ok, sc, 1.0), g.shape)), 0)
    return codes.reshape(f.shape).astype(np.uint8), bits


def rope_rows(k, positions, rope_theta, rope_style=oracle.ROPE_NEOX):
    """The rotation in fp64, rounded to float32 and then to the storage type."""
    if rope_style == oracle.ROPE_NONE:
        return k
    f = oracle.to_f64(k)
    y = np.array([[oracle.rope(f[t, h], int(positions[t]), rope_theta, rope_style) for h in range(k.shape[1])]
                  for t in range(k.shape[0])]).astype(np.float32).reshape(k.shape)
    if k.dtype == np.float32:
        return y
    return np.array([oracle.round_bf16(x) for x in y.ravel().tolist()], np.uint16).reshape(k.shape)


def record_positions(d: int):
    """(code byte [2][16][d], nibble [d], scale byte [2][16][d / 64]) of K (0) and V (1)."""
    byte = np.zeros((2, 16, d), np.int64)
    scale = np.zeros((2, 16, d // GROUP), np.int64)
    for r in range(16):
        quad, rest = divmod(r, 4)
        frag, j = divmod(rest, 2)
        for e in range(d):
            plane, x = divmod(e, 64)
            byte[0, r, e] = 512 * plane + 16 * (4 * (2 * quad + j) + x // 16) + 8 * frag + (x % 16) // 2
            byte[1, r, e] = 8 * d + 512 * plane + 16 * (4 * (x // 8) + quad) + 4 * rest + (x % 8) // 2
        for hh in range(d // GROUP):
            for w in range(2):
                scale[w, r, hh] = 16 * d + 64 * hh + 16 * quad + 8 * w + 2 * rest
    return byte, np.arange(d) & 1, scale


def write(k, v, positions, slots, pool, rope_theta, rope_style=oracle.ROPE_NEOX):
    """In-place 4-bit write of storage rows k, v [T, H, d] into pool uint8 [nb, H, 17 d]."""
    k = rope_rows(k, positions, rope_theta, rope_style)
    T, H, d = k.shape
    byte, nib, sb = record_positions(d)
    for w, x in enumerate((k, v)):
        codes, bits = quantise(x)
        for t in range(T):
            if slots[t] < 0:
                continue
            b, r = divmod(int(slots[t]), 16)
            for h in range(H):
                rec = pool[b, h]
                rec[byte[w, r, 0::2]] = codes[t, h, 0::2] | (codes[t, h, 1::2] << 4)
                rec[sb[w, r]] = bits[t, h] & 0xFF
                rec[sb[w, r] + 1] = bits[t, h] >> 8


def dequant(pool, d):
    """fp64 K and V [nb, H, 16, d] of a 4-bit pool."""
    byte, nib, sb = record_positions(d)
    out = []
    for w in range(2):
        codes = (pool[:, :, byte[w]] >> (4 * nib)) & 15
        bits = pool[:, :, sb[w]].astype(np.uint16) | (pool[:, :, sb[w] + 1].astype(np.uint16) << 8)
        out.append(VALUES[codes] * np.repeat(oracle.bf16_to_f64(bits), GROUP, axis=-1))
    return out


def paged_attention(q, pool, block_tables, context_lens, scale):
    """Decode attention over the exactly dequantised values, fp64 [B, H_q, d]."""
    kd, vd = (np.ascontiguousarray(x) for x in dequant(pool, q.shape[-1]))
    return oracle.paged_attention(np.ascontiguousarray(oracle.to_f64(q)), kd, vd, block_tables, context_lens, scale)


def step_metadata(nc, nn, tables, stack, max_tokens, num_blocks):
    """The device step's definition over plain lists: (tables, stack, lists of
    token_seq / positions / slots padded to max_tokens, contexts, status).
    tables int array [B, W] and stack (list, last entry next) are not changed."""
    bt, st = np.array(tables), list(stack)
    B, W = bt.shape
    bad = len(st) > num_blocks
    tokens = blocks = 0
    for c, n in zip(nc, nn):
        have, need = -(-int(c) // 16), -(-(int(c) + int(n)) // 16)
        bad |= c < 0 or int(c) + int(n) > 2 ** 31 - 1 or have > W or (n >= 0 and need > W)
        tokens += max(int(n), 0)
        blocks += need - have if n >= 0 else 0
    released = sum(-(-int(c) // 16) for c, n in zip(nc, nn) if n < 0 and c >= 0)
    for s in range(B if not bad else 0):        # what goes back to the pool must come from it
        if nn[s] < 0:
            bad |= any(not 0 <= int(x) < num_blocks for x in bt[s, :-(-int(nc[s]) // 16)])
    bad |= tokens > max_tokens or len(st) + released > num_blocks
    status = -1 if bad else (-5 if blocks > len(st) + released else 0)
    seq, pos, slots = [], [], []
    ctx = np.zeros(B, np.int32)
    if status == 0:
        for s in range(B):
            if nn[s] < 0:
                h = -(-int(nc[s]) // 16)
                st += [int(x) for x in bt[s, :h]]
                bt[s, :h] = -1
        for s in range(B):
            if nn[s] < 0:
                continue
            for i in range(-(-int(nc[s]) // 16), -(-(int(nc[s]) + int(nn[s])) // 16)):
                bt[s, i] = st.pop()
            ctx[s] = nc[s] + nn[s]
            for p in range(int(nc[s]), int(ctx[s])):
                seq.append(s)
                pos.append(p)
                b = int(bt[s, p // 16])
                slots.append(b * 16 + p % 16 if 0 <= b < num_blocks else -1)
    pad = max_tokens - len(seq)
    return bt, st, seq + [0] * pad, pos + [-1] * pad, slots + [-1] * pad, ctx, status
