"""Workloads of the q/k norms fused with rotation and cache write, and of the
8-bit KV cache with a scale per block and head.

Four operators, each with a plain form (elementary torch operations) and the
library's calls (`own`):

  norm    photon_qk_norm_rope_kv_cache_write: RMS norms of a step's queries and
          keys per head, their rotation, and the write of keys and values
  write   photon_kv_cache_write_int8, or with norms
          photon_qk_norm_rope_kv_cache_write_int8: the same into 8-bit pages,
          read back with photon_kv_cache_read_int8
  read    photon_kv_cache_read_int8: cached tokens as bf16 (a prefix that is
          attended to by a prefill)
  decode  photon_paged_attention_decode_int8: attention of one query token per
          sequence over the 8-bit pages

The 8-bit pool is uint8 [num_blocks][kv_heads][32 d + 16]: per (block of 16
tokens, KV head) one record of K codes, V codes and one fp32 scale each for K
and V.  value = (byte - 128) * scale.  Byte positions are those of
`record_layout`.

A write takes m, the largest magnitude of the rows that it writes to a block
(K and V apart).  A call that writes a block's first token starts it anew: its
other rows become zero, its old scale does not count.  The scale s stays where
fl(m / 127) does not exceed it and becomes max(fl(m / 127), 2 s) where it does;
the kept rows' codes are then rounded to the new scale.  A new code is y / s
rounded to nearest even, the division being a product with fl(1 / s).
"""
import functools
import math
import random

import torch

own = False

DEVICE = "cuda"
BLOCK = 16     # tokens of a page
LOST = 2.0 ** -100   # smaller scales count as zero


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # the new tokens of a 64-sequence decode step, 16 query and 8 KV heads of 128
        dict(name="norm_decode64", op="norm", tokens=64, kv_heads=8, group=2, head_dim=128, run=1,
             dtype="bf16", rope="neox", theta=1e6),
        # four 2048-token prompts, 32 query and 8 KV heads of 64
        dict(name="norm_prompts8192", op="norm", tokens=8192, kv_heads=8, group=4, head_dim=64, run=2048,
             dtype="bf16", rope="neox", theta=5e5),
        # an odd chunk in 32 bits with interleaved rotation
        dict(name="norm_f32_chunk777", op="norm", tokens=777, kv_heads=4, group=1, head_dim=128, run=111,
             dtype="f32", rope="gptj", theta=1e4),
        # a 64-sequence decode step into 8 bits, with the norms
        dict(name="write_decode64", op="write", tokens=64, kv_heads=8, group=2, head_dim=128, run=1,
             dtype="bf16", rope="neox", theta=1e6, norm=True),
        # eight 2048-token prompts into 8 bits, 8 KV heads of 64
        dict(name="write_prompts16384", op="write", tokens=16384, kv_heads=8, group=4, head_dim=64, run=2048,
             dtype="bf16", rope="neox", theta=5e5, norm=False),
        # an odd chunk of 32-bit keys and values
        dict(name="write_f32_chunk777", op="write", tokens=777, kv_heads=4, group=2, head_dim=128, run=111,
             dtype="f32", rope="gptj", theta=1e4, norm=False),
        # a short shared prefix
        dict(name="read_prefix101", op="read", tokens=101, kv_heads=8, head_dim=64, run=101),
        # the prefixes of a large prompt batch
        dict(name="read_prefix32768", op="read", tokens=32768, kv_heads=8, head_dim=128, run=4096),
        # one request, 1024 tokens of context: latency
        dict(name="decode_single1024", op="decode", seqs=1, kv_heads=8, group=4, head_dim=64,
             shape="equal", lo=1024, hi=1024, partition=32, out="bf16"),
        # a ragged batch with heads of 128
        dict(name="decode_ragged64", op="decode", seqs=64, kv_heads=8, group=2, head_dim=128,
             shape="lognormal", lo=16, hi=8192, partition=128, out="bf16"),
        # few long sequences, wide query groups, 32-bit output
        dict(name="decode_long8_f32", op="decode", seqs=8, kv_heads=4, group=8, head_dim=128,
             shape="uniform", lo=8192, hi=32768, partition=256, out="f32"),
        # long contexts, some of one token and some empty
        dict(name="decode_long128", op="decode", seqs=128, kv_heads=8, group=4, head_dim=64,
             shape="uniform", lo=512, hi=32768, partition=512, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "write", "read", "decode"))
    if op != "decode":
        tokens = _log(rng, 1, 16384)
        case = dict(op=op, tokens=tokens, kv_heads=rng.choice((1, 2, 3, 4, 8)),
                    head_dim=rng.choice((32, 64, 128, 256) if op == "norm" else (64, 128)),
                    run=max(1, tokens // rng.randint(1, 32)))
        if tokens > 8192 and case["kv_heads"] * case["head_dim"] > 512:
            case["kv_heads"] = max(1, 512 // case["head_dim"])
        if op != "read":
            case.update(group=rng.choice((1, 2, 4)), dtype=rng.choice(("bf16", "bf16", "f32")),
                        rope=rng.choice(("neox", "neox", "gptj", "none")), theta=rng.choice((1e4, 5e5, 1e6)))
        if op == "write":
            case.update(norm=rng.random() < 0.5)
        return case
    heads, group = rng.choice(((8, 4), (8, 2), (8, 1), (4, 8), (2, 4), (1, 8)))
    seqs = _log(rng, 1, 128)
    hi = _log(rng, 16, 32768)
    return dict(op=op, seqs=seqs, kv_heads=heads, group=group, head_dim=rng.choice((64, 128)) if seqs <= 64 else 64,
                shape=rng.choice(("uniform", "lognormal", "equal")), lo=max(1, hi // 16), hi=hi,
                partition=rng.choice((32, 64, 128, 256, 512)), out=rng.choice(("bf16", "bf16", "f32")))


# ---- the 8-bit record ---------------------------------------------------------

def record_bytes(d):
    return 2 * BLOCK * d + 16


@functools.lru_cache(maxsize=None)
def record_layout(d, device):
    """Byte offsets in a record of the K and the V codes [2, 16, d], in planes
    of 64 dims.  K: the row of token 4a + 2n + j is row 8n + 2a + j.  V: 8
    consecutive dims of a token, then those of its neighbour (token ^ 1), the
    tokens 4c .. 4c + 1 of c = 0..3 next to each other, likewise 4c + 2 .. 4c + 3."""
    r = torch.arange(BLOCK)[:, None]
    e = torch.arange(d)[None, :]
    k = (e // 64) * 1024 + (8 * ((r >> 1) & 1) + 2 * (r // 4) + (r & 1)) * 64 + e % 64
    v = 16 * d + (e // 64) * 1024 + ((r >> 1) & 1) * 512 + ((e % 64 // 8) * 4 + r // 4) * 16 + (r & 1) * 8 + e % 8
    return torch.stack([k, v]).to(device)


def scales(pool):
    """[blocks, heads, 2] fp32 view of a pool's K and V scales."""
    n = pool.shape[-1] // 4
    return pool.view(torch.float32)[..., n - 4:n - 2]


def load(rec, d, which):
    """Values [..., 16, d] (fp32) of K (which 0) or V (1) of records [..., bytes]."""
    code = rec[..., record_layout(d, rec.device)[which]].float() - 128
    return code * scales(rec)[..., which][..., None, None]


def load_rows(pool, slots, d, which):
    """Values [T, H, d] (fp32) of the tokens at `slots`."""
    blk, off = slots // BLOCK, slots % BLOCK
    h = torch.arange(pool.shape[1], device=pool.device)[None, :, None]
    at = record_layout(d, pool.device)[which][off][:, None, :]
    return (pool[blk[:, None, None], h, at].float() - 128) * scales(pool)[blk][..., which][..., None]


def store(pool, slots, y, which):
    """Writes rows y [T, H, d] (64 bits) of K (which 0) or V (1) to `slots`."""
    d, dev = y.shape[-1], pool.device
    blk, off = slots // BLOCK, slots % BLOCK
    anew = torch.zeros(len(pool), dtype=torch.int32, device=dev).index_add(0, blk, (off == 0).int())[:, None] > 0
    old = torch.where(anew, 0.0, scales(pool)[..., which])                                # [blocks, H]
    top = torch.zeros_like(old, dtype=torch.float64)
    top = top.scatter_reduce(0, blk[:, None].expand(-1, y.shape[1]), y.abs().amax(-1), "amax")
    want = (top / 127).float()
    want = torch.where(want < LOST, 0.0, want)
    new = torch.where(want > old, torch.maximum(want, 2 * old), old)
    inv = torch.where(new > 0, 1 / torch.where(new > 0, new, 1.0), 0.0)
    ratio = torch.where(new > old, old * inv, 1.0)
    at = record_layout(d, dev)[which]
    codes = pool[..., at].float() - 128                                                   # [blocks, H, 16, d]
    codes = torch.where(anew[..., None, None], 0.0, (codes * ratio[..., None, None]).round())
    codes[blk, :, off] = (y * inv[blk][..., None].double()).round().float()
    pool[..., at] = (codes + 128).to(torch.uint8)
    scales(pool)[..., which] = new


# ---- inputs -------------------------------------------------------------------

def _pool(gen, blocks, heads, d, std=0.5):
    """A pool whose pages hold quantised normal values: a bank of 256 pages,
    one drawn for each (block, head)."""
    bank = torch.zeros(256, 1, record_bytes(d), dtype=torch.uint8, device=DEVICE)
    every = torch.arange(256 * BLOCK, device=DEVICE)
    for which in (0, 1):
        x = torch.randn(256 * BLOCK, 1, d, generator=gen, device=DEVICE) * std
        store(bank, every, x.double(), which)
    pick = torch.randint(0, 256, (blocks * heads,), generator=gen, device=DEVICE)
    return bank[:, 0][pick].view(blocks, heads, -1)


def _contexts(case, seed):
    rng = random.Random(seed)
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    if case["shape"] == "equal":
        return [hi] * n
    if case["shape"] == "lognormal":
        mid = math.sqrt(lo * hi) if lo * 64 > hi else 1500
        lens = [min(hi, max(lo, round(rng.lognormvariate(math.log(mid), 0.8)))) for _ in range(n)]
    else:
        lens = [rng.randint(lo, hi) for _ in range(n)]
    for s in range(0, n, 43):        # about 2 % of one token, 2 % empty (n > 20)
        if n > 20:
            lens[s], lens[(s + 21) % n] = 1, 0
    return lens


def _slots(gen, tokens, run):
    """Slots of `tokens` tokens: runs of consecutive positions, each from an
    offset of its own in its first block, over shuffled blocks."""
    runs = -(-tokens // run)
    per = -(-run // BLOCK) + 1
    blocks = int(runs * per * 1.25) + 1
    perm = torch.randperm(blocks, generator=gen, device=DEVICE)
    start = torch.randint(0, BLOCK, (runs,), generator=gen, device=DEVICE)
    t = torch.arange(tokens, device=DEVICE)
    pos = start[t // run] + t % run
    first = perm[torch.arange(runs, device=DEVICE) * per]
    return blocks, perm[(t // run) * per + pos // BLOCK] * BLOCK + pos % BLOCK, pos, first


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(int(seed) * 7919 + 17)
    op, d, H = case["op"], case["head_dim"], case["kv_heads"]
    s = dict(op=op, case=case)
    if op != "decode":
        T = case["tokens"]
        blocks, slots, pos, first = _slots(gen, T, case["run"])
        if op == "read":
            s.update(pool=_pool(gen, blocks, H, d), slots=slots.contiguous())
            s.update({n: torch.empty(T, H, d, dtype=torch.bfloat16, device=DEVICE) for n in ("k_out", "v_out")})
            return s
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        if case["run"] == 1:      # decode tokens: positions anywhere in their sequences
            pos = pos + BLOCK * torch.randint(0, 512, (T,), generator=gen, device=DEVICE)
        k, v = (torch.randn(T, H, d, generator=gen, device=DEVICE) * 0.5 for _ in range(2))
        q = torch.randn(T, H * case["group"], d, generator=gen, device=DEVICE) * 0.5
        wq, wk = (1 + 0.2 * torch.randn(d, generator=gen, device=DEVICE) for _ in range(2))
        s.update(k=k.to(dt), v=v.to(dt), q=q.to(dt), q_weight=wq.to(dt), k_weight=wk.to(dt), eps=1e-6,
                 slots=slots.contiguous(), pos=pos.int().contiguous())
        if op == "norm":
            s.update({n: torch.zeros(blocks, H, BLOCK, d, dtype=dt, device=DEVICE) for n in ("k_cache", "v_cache")})
            return s
        # what is read back: every written token, and all rows of the blocks that the runs begin in
        rest = first[:, None] * BLOCK + torch.arange(BLOCK, device=DEVICE)
        back = torch.cat([slots, rest.flatten()]).contiguous()
        s.update(pool=_pool(gen, blocks, H, d), back=back)
        s.update({n: torch.empty(len(back), H, d, dtype=torch.bfloat16, device=DEVICE) for n in ("k_out", "v_out")})
        return s
    lens = _contexts(case, seed)
    B, G = case["seqs"], case["group"]
    W = max(1, -(-max(lens) // BLOCK))
    pages = [-(-c // BLOCK) for c in lens]
    blocks = int(sum(pages) * 1.05) + 1
    need = torch.tensor(pages, device=DEVICE)
    perm = torch.randperm(blocks, generator=gen, device=DEVICE).int()
    col = torch.arange(W, device=DEVICE)[None, :]
    at = (need.cumsum(0) - need)[:, None] + col
    tables = torch.where(col < need[:, None], perm[at.clamp(max=blocks - 1)], -1).contiguous()
    dt = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    s.update(pool=_pool(gen, blocks, H, d), tables=tables, max_len=W * BLOCK, scale=d ** -0.5,
             lens=torch.tensor(lens, dtype=torch.int32, device=DEVICE),
             q=(torch.randn(B, H * G, d, generator=gen, device=DEVICE) * 0.5).to(torch.bfloat16),
             out=torch.empty(B, H * G, d, dtype=dt, device=DEVICE))
    # the split-K workspace a program keeps: per (sequence, query head) one slot
    # more than the partitions, each a maximum, a sum and a row of output
    part = -(-W * BLOCK // case["partition"]) + 1
    rows = B * H * G
    s["workspace"] = torch.empty(4 * rows * part * (d + 2) + 8 * rows + 4096, dtype=torch.uint8, device=DEVICE)
    return s


# ---- one pass -------------------------------------------------------------------

def _normed(x, w, eps):
    """RMS norm of rows [T, H, d] in 64 bits: what follows may round at a border."""
    x = x.double()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()


def _rotate(x, pos, style, theta):
    """RoPE of x [T, H, d] in 64 bits: far positions have large angles."""
    x, d = x.double(), x.shape[-1]
    if style == "none":
        return x
    freq = theta ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device=x.device) / d)
    ang = pos.double()[:, None, None] * freq
    c, n = ang.cos(), ang.sin()
    a, b = (x[..., 0::2], x[..., 1::2]) if style == "gptj" else (x[..., :d // 2], x[..., d // 2:])
    y = (a * c - b * n, b * c + a * n)
    return torch.stack(y, -1).flatten(-2) if style == "gptj" else torch.cat(y, -1)


def _norm_plain(s):
    c = s["case"]
    k = _rotate(_normed(s["k"], s["k_weight"], s["eps"]), s["pos"], c["rope"], c["theta"])
    blk, off = s["slots"] // BLOCK, s["slots"] % BLOCK
    s["k_cache"][blk, :, off] = k.to(s["k_cache"].dtype)
    s["v_cache"][blk, :, off] = s["v"]
    s["q"].copy_(_rotate(_normed(s["q"], s["q_weight"], s["eps"]), s["pos"], c["rope"], c["theta"]))


def _write_plain(s):
    c, k = s["case"], s["k"]
    if c["norm"]:
        k = _normed(k, s["k_weight"], s["eps"])
        s["q"].copy_(_rotate(_normed(s["q"], s["q_weight"], s["eps"]), s["pos"], c["rope"], c["theta"]))
    store(s["pool"], s["slots"], _rotate(k, s["pos"], c["rope"], c["theta"]), 0)
    store(s["pool"], s["slots"], s["v"].double(), 1)


def _read_plain(s, slots):
    for which, out in ((0, s["k_out"]), (1, s["v_out"])):
        out.copy_(load_rows(s["pool"], slots, out.shape[-1], which))


def _decode_plain(s):
    c = s["case"]
    d, H, G = c["head_dim"], c["kv_heads"], c["group"]
    rec = s["pool"][s["tables"].clamp(min=0).long()].transpose(1, 2).contiguous()   # [B, H, W, bytes]
    q = s["q"].float().unflatten(1, (H, G))                                         # [B, H, G, d]
    p = q @ load(rec, d, 0).flatten(2, 3).transpose(-1, -2) * s["scale"]
    n = torch.arange(p.shape[-1], device=p.device)
    p = p.masked_fill(n >= s["lens"].view(-1, 1, 1, 1), -math.inf)
    top = p.amax(-1, keepdim=True)
    p = (p - torch.where(top.isinf(), 0.0, top)).exp()
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    s["out"].copy_((p @ load(rec, d, 1).flatten(2, 3)).flatten(1, 2))


def run(s):
    op, c = s["op"], s["case"]
    if own:
        import paged_kv_decode_write_gb300 as pk
        if op == "norm":
            pk.photon_qk_norm_rope_kv_cache_write(
                s["q"], s["pos"], s["k"], s["v"], s["pos"], s["slots"], s["q_weight"], s["k_weight"], s["eps"],
                s["k_cache"], s["v_cache"], c["theta"], c["rope"])
        elif op == "decode":
            pk.photon_paged_attention_decode_int8(s["q"], s["pool"], s["tables"], s["lens"], s["scale"], s["out"],
                                                  s["max_len"], c["partition"], s["workspace"])
        elif op == "read":
            pk.photon_kv_cache_read_int8(s["pool"], s["slots"], s["k_out"], s["v_out"])
        else:
            if c["norm"]:
                pk.photon_qk_norm_rope_kv_cache_write_int8(
                    s["q"], s["pos"], s["k"], s["v"], s["pos"], s["slots"], s["q_weight"], s["k_weight"], s["eps"],
                    s["pool"], c["theta"], c["rope"])
            else:
                pk.photon_kv_cache_write_int8(s["k"], s["v"], s["pos"], s["slots"], s["pool"], c["theta"], c["rope"])
            pk.photon_kv_cache_read_int8(s["pool"], s["back"], s["k_out"], s["v_out"])
    elif op == "norm":
        _norm_plain(s)
    elif op == "decode":
        _decode_plain(s)
    elif op == "read":
        _read_plain(s, s["slots"])
    else:
        _write_plain(s)
        _read_plain(s, s["back"])
    if op == "norm":
        return [s["q"], s["k_cache"], s["v_cache"]]
    if op == "decode":
        return [s["out"]]
    return [s["k_out"], s["v_out"]] + ([s["q"]] if op == "write" and c["norm"] else [])


def work(case):
    op, d, H = case["op"], case["head_dim"], case["kv_heads"]
    token = H * record_bytes(d) / BLOCK            # 8-bit bytes of a token's K and V
    if op == "read":
        T = case["tokens"]
        return dict(bytes=T * (token + 2 * H * d * 2 + 8), flops=0.0)
    if op in ("norm", "write"):
        T, size = case["tokens"], 2 if case["dtype"] == "bf16" else 4
        queries = 2 * T * H * case["group"] * d * size
        if op == "norm":                           # k and v in and out, q in and out
            return dict(bytes=T * (4 * H * d * size + 16) + queries, flops=0.0)
        back = T + BLOCK * -(-T // case["run"])    # tokens read back
        return dict(bytes=T * (2 * H * d * size + token + 12) + back * (token + 2 * H * d * 2 + 8)
                    + (queries + 4 * T if case["norm"] else 0), flops=0.0)
    lens = _contexts(case, 0)
    total, rows = sum(lens), case["seqs"] * H * case["group"]
    size = 2 if case["out"] == "bf16" else 4
    return dict(bytes=total * token + rows * d * (2 + size) + 4.0 * sum(-(-c // BLOCK) for c in lens),
                flops=4.0 * total * H * case["group"] * d)


# ---- the definition in 64 bits ------------------------------------------------------

def _values64(rec, d, which):
    """Values [..., 16, d] (fp64) of records' K or V, and their scales [...]."""
    tok = torch.arange(BLOCK, device=rec.device)
    a, n, j = tok // 4, tok // 2 % 2, tok % 2
    planes = []
    for hh in range(d // 64):
        at = (16 * d if which else 0) + 1024 * hh
        raw = rec[..., at:at + 1024]
        if which == 0:       # rows (n, a, j) of 64 dims
            planes.append(raw.unflatten(-1, (2, 4, 2, 64))[..., n, a, j, :])
        else:                # (n, dims / 8, a, j, dims % 8)
            planes.append(raw.unflatten(-1, (2, 8, 4, 2, 8)).movedim(-4, -2)[..., n, a, j, :, :].flatten(-2))
    raw = rec[..., 32 * d + 4 * which:32 * d + 4 * which + 4].long()
    bits = raw[..., 0] | raw[..., 1] << 8 | raw[..., 2] << 16 | raw[..., 3] << 24
    scale = bits.to(torch.int32).view(torch.float32).double()
    return (torch.cat(planes, -1).double() - 128) * scale[..., None, None], scale


def _turned(x, w, eps, pos, style, theta):
    """Norm (w given) and rotation in 64 bits, pairs as complex numbers."""
    x, d = x.double(), x.shape[-1]
    if w is not None:
        x = w.double() * x / (x.square().sum(-1, keepdim=True) / d + eps).sqrt()
    if style == "none":
        return x
    i = torch.arange(d // 2, dtype=torch.float64, device=x.device)
    turn = pos.double()[:, None] * torch.exp(i * (-2 * math.log(theta) / d))
    z = x.unflatten(-1, (-1, 2)) if style == "gptj" else x.unflatten(-1, (2, -1)).transpose(-1, -2)
    z = torch.view_as_complex(z.contiguous()) * torch.polar(torch.ones_like(turn), turn)[:, None]
    z = torch.view_as_real(z)
    return z.flatten(-2) if style == "gptj" else z.transpose(-1, -2).flatten(-2)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    d, H = case["head_dim"], case["kv_heads"]
    if op == "decode":
        G = case["group"]
        out = torch.zeros(case["seqs"], H * G, d, dtype=torch.float64, device=DEVICE)
        for b, n in enumerate(s["lens"].tolist()):
            if n:
                rec = s["pool"][s["tables"][b, :-(-n // BLOCK)].long()].transpose(0, 1)
                k, v = (_values64(rec, d, w)[0].flatten(1, 2)[:, :n] for w in (0, 1))
                q = s["q"][b].double().view(H, G, d)
                out[b] = (torch.softmax(q @ k.mT * s["scale"], -1) @ v).view(H * G, d)
        return [out]
    if op == "read":
        blk, off = s["slots"] // BLOCK, s["slots"] % BLOCK
        step, got = 2048, ([], [])
        for t in range(0, len(blk), step):
            rec, o = s["pool"][blk[t:t + step]], off[t:t + step]
            for w in (0, 1):
                got[w].append(_values64(rec, d, w)[0][torch.arange(len(o), device=DEVICE), :, o])
        return [torch.cat(g) for g in got]
    style, theta, eps = case["rope"], case["theta"], s["eps"]
    normed = op == "norm" or case["norm"]
    q = _turned(s["q"], s["q_weight"], eps, s["pos"], style, theta)
    k = _turned(s["k"], s["k_weight"] if normed else None, eps, s["pos"], style, theta)
    if op == "norm":
        caches = []
        for x in (k, s["v"].double()):
            flat = torch.zeros(s["k_cache"].shape[0] * BLOCK, H, d, dtype=torch.float64, device=DEVICE)
            flat[s["slots"]] = x
            caches.append(flat.view(-1, BLOCK, H, d).transpose(1, 2).contiguous())
        return [q] + caches
    # per block a dense [16] of which token each row gets, or none
    blocks = s["pool"].shape[0]
    token = torch.full((blocks * BLOCK,), -1, device=DEVICE)
    token[s["slots"]] = torch.arange(len(s["slots"]), device=DEVICE)
    token = token.view(blocks, BLOCK)
    res, step = [], 1024
    for w, x in ((0, k), (1, s["v"].double())):
        rows = []
        for b in range(0, blocks, step):
            tok = token[b:b + step]
            fresh, given = tok[:, 0] >= 0, (tok >= 0)[:, :, None, None]
            y = torch.where(given, x[tok.clamp(min=0)], 0.0).transpose(1, 2)             # [b, H, 16, d]
            old, scale = _values64(s["pool"][b:b + step], d, w)
            scale = torch.where(fresh[:, None], 0.0, scale)
            code = torch.where(fresh[:, None, None, None], 0.0, old / scale.clamp(min=1e-300)[..., None, None]).round()
            need = (y.abs().amax((-1, -2)) / 127).float().double()
            need = torch.where(need < LOST, 0.0, need)
            new = torch.where(need <= scale, scale, torch.maximum(need, 2 * scale))
            inv = torch.where(new > 0, (1 / new).float().double(), 0.0)
            kept = torch.where((new == scale)[..., None, None], code, (code * (scale * inv).float().double()[..., None, None]).round())
            mine = (y * inv[..., None, None]).round()
            rows.append((torch.where(given.transpose(1, 2), mine, kept) * new[..., None, None]).transpose(1, 2).flatten(0, 1))
        res.append(torch.cat(rows)[s["back"]])
    return res + ([q] if normed else [])
