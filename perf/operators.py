"""Workloads of the 4-bit KV cache and of the step metadata built on the GPU.

Four operators, each with a plain form (elementary torch operations) and the
library's calls (`own`):

  metadata  photon_build_step_metadata_device: token, position and slot lists,
            context lengths and grown block tables of one scheduler step, from
            the requests' lengths, with a free list that lives on the GPU
  write     photon_kv_cache_write_fp4: RoPE, 4-bit quantisation and scatter of
            a step's keys and values, read back with photon_kv_cache_read_fp4
  read      photon_kv_cache_read_fp4: gather and dequantisation of cached
            tokens (a prefix that is attended to in bf16)
  decode    photon_paged_attention_decode_fp4: attention of one query token
            per sequence over the 4-bit pages

The 4-bit pool is uint8 [num_blocks][kv_heads][1088 * d / 64]: per (block, KV
head) one record of K codes, V codes and scales for 16 tokens.  A
code is E2M1 (sign, two exponent bits, one mantissa bit: 0, .5, 1, 1.5, 2, 3,
4, 6); each token has one bf16 scale per 64 head dims.  Byte positions inside
a record are those of `record_layout`.
"""
import functools
import math
import random

import torch

own = False

BLOCK = 16     # tokens of a page
GROUP = 64     # head dims that share a scale
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # the running requests of a 64-sequence decode step: one token each
        dict(name="metadata_decode64", op="metadata", seqs=64, width=512, prompts=0.0,
             prompt_median=1, context_median=1500, max_tokens=64),
        # a large batch with freshly admitted prompts among running requests
        dict(name="metadata_mixed2048", op="metadata", seqs=2048, width=512, prompts=0.25,
             prompt_median=96, context_median=1500, max_tokens=65536),
        # the new tokens of a 64-sequence decode step, 8 KV heads of 128
        dict(name="write_decode64", op="write", tokens=64, kv_heads=8, head_dim=128, run=1,
             dtype="bf16", rope="neox", theta=1e6),
        # eight 2048-token prompts, 8 KV heads of 64
        dict(name="write_prompts16384", op="write", tokens=16384, kv_heads=8, head_dim=64,
             run=2048, dtype="bf16", rope="neox", theta=5e5),
        # an odd chunk of 32-bit keys and values with interleaved rotation
        dict(name="write_f32_chunk777", op="write", tokens=777, kv_heads=4, head_dim=128, run=111,
             dtype="f32", rope="gptj", theta=1e4),
        # a short shared prefix
        dict(name="read_prefix101", op="read", tokens=101, kv_heads=8, head_dim=64, run=101,
             dtype="bf16"),
        # the prefixes of a large prompt batch, brought back to bf16
        dict(name="read_prefix32768", op="read", tokens=32768, kv_heads=8, head_dim=128, run=4096,
             dtype="bf16"),
        # one request, 1024 tokens of context: latency
        dict(name="decode_single1024", op="decode", seqs=1, kv_heads=8, group=4, head_dim=64,
             shape="equal", lo=1024, hi=1024, partition=32, out="bf16"),
        # a small continuous batch
        dict(name="decode_batch16", op="decode", seqs=16, kv_heads=8, group=4, head_dim=64,
             shape="uniform", lo=100, hi=2048, partition=64, out="bf16"),
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
    op = rng.choice(("metadata", "write", "read", "decode"))
    if op == "metadata":
        seqs = _log(rng, 1, 2048)
        prompts = rng.choice((0.0, 0.1, 0.5, 1.0))
        tokens = seqs if prompts == 0.0 else min(65536, seqs + _log(rng, 16, 65536))
        return dict(op=op, seqs=seqs, width=rng.randint(64, 512), prompts=prompts,
                    prompt_median=_log(rng, 8, 512), context_median=_log(rng, 16, 4096),
                    max_tokens=tokens)
    if op in ("write", "read"):
        tokens = _log(rng, 1, 16384)
        case = dict(op=op, tokens=tokens, kv_heads=rng.choice((1, 2, 4, 8)),
                    head_dim=rng.choice((64, 128)), run=max(1, tokens // rng.randint(1, 32)),
                    dtype=rng.choice(("bf16", "bf16", "f32")))
        if op == "write":
            if tokens > 8192 and case["kv_heads"] * case["head_dim"] > 512:
                case["kv_heads"] = 512 // case["head_dim"]
            case.update(rope=rng.choice(("neox", "neox", "gptj", "none")),
                        theta=rng.choice((1e4, 5e5, 1e6)))
        return case
    heads, group = rng.choice(((8, 4), (8, 2), (8, 1), (4, 8), (2, 4), (1, 8)))
    seqs = _log(rng, 1, 128)
    hi = _log(rng, 16, 32768)
    return dict(op=op, seqs=seqs, kv_heads=heads, group=group, head_dim=rng.choice((64, 128)) if seqs <= 64 else 64,
                shape=rng.choice(("uniform", "lognormal", "equal")), lo=max(1, hi // 16), hi=hi,
                partition=rng.choice((32, 64, 128, 256, 512)), out=rng.choice(("bf16", "bf16", "f32")))


# ---- the 4-bit record ---------------------------------------------------------

def record_bytes(d):
    return 2 * BLOCK * d // 2 + 2 * BLOCK * (d // GROUP) * 2


@functools.lru_cache(maxsize=None)
def record_layout(d, device):
    """Byte offsets in a record: K codes [16, d/2] (low nibble: the even dim),
    V codes [16, d/2] (the same), and the first bytes of the K and V scales
    [16, d/64].  Codes lie in planes of 512 bytes, one per 64 dims.  K: token
    4c + 2n + j sits with column 2c + j of fragment n, 16 consecutive dims to
    a lane.  V: a token's 8 consecutive dims are one 32-bit word, the words of
    four consecutive tokens one 16-byte chunk.  Scales: per 64 dims and four
    consecutive tokens a chunk of their four K and four V scales."""
    r = torch.arange(BLOCK)[:, None]
    e = 2 * torch.arange(d // 2)[None, :]
    col, n = 2 * (r // 4) + (r & 1), (r // 2) & 1
    k = (e // 64) * 512 + (4 * col + (e % 64) // 16) * 16 + n * 8 + (e % 16) // 2
    v = 8 * d + (e // 64) * 512 + (((e % 64) // 8) * 4 + r // 4) * 16 + (r & 3) * 4 + (e % 8) // 2
    s = 16 * d + 64 * torch.arange(d // GROUP)[None, :] + 16 * (r // 4) + 2 * (r % 4)
    return k.to(device), v.to(device), s.to(device), (s + 8).to(device)


@functools.lru_cache(maxsize=None)
def byte_values(device):
    """[256, 2]: the values of a byte's low and high code."""
    m = torch.tensor(MAGNITUDES)
    one = torch.cat([m, -m])
    b = torch.arange(256)
    return torch.stack([one[b & 15], one[b >> 4]], 1).to(device)


def quantise(x):
    """Codes and bf16 scales of x [..., d]: per 64 dims, scale = bf16(max|x| / 6),
    code = the nearest E2M1 of x / scale, halves to the even code (|x| against
    the midpoints times the scale, products that 32 bits hold exactly)."""
    g = x.float().unflatten(-1, (-1, GROUP))
    scale = (g.abs().amax(-1) / 6).to(torch.bfloat16)
    m, s = g.abs(), scale[..., None].float()
    code = ((m > 0.25 * s).to(torch.uint8) + ((m >= 0.75 * s) & (m > 0)) + (m > 1.25 * s)
            + ((m >= 1.75 * s) & (m > 0)) + (m > 2.5 * s) + ((m >= 3.5 * s) & (m > 0)) + (m > 5.0 * s))
    code = torch.where(s > 0, code, 0).to(torch.uint8)
    code = torch.where(g < 0, code + 8, code).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def store(pool, blk, off, codes, scales, which):
    """Scatters [T, H, d/2] code bytes and [T, H, d/64] scales of K (which 0) or V (1)."""
    d = codes.shape[-1] * 2
    at, at_s = record_layout(d, pool.device)[which], record_layout(d, pool.device)[2 + which]
    h = torch.arange(codes.shape[1], device=pool.device)[None, :, None]
    pool[blk[:, None, None], h, at[off][:, None, :]] = codes
    raw = scales.contiguous().view(torch.uint8).unflatten(-1, (-1, 2))
    two = torch.arange(2, device=pool.device)
    pool[blk[:, None, None, None], h[..., None], at_s[off][:, None, :, None] + two] = raw


def load(rec, d, which, at=slice(None)):
    """Values [..., rows, d] (fp32) of K (which 0) or V (1) of records [..., bytes]."""
    lay = record_layout(d, rec.device)
    codes = rec[..., lay[which][at]]
    two = torch.arange(2, device=rec.device)
    scale = rec[..., lay[2 + which][at][..., None] + two].view(torch.bfloat16).squeeze(-1)
    x = byte_values(rec.device)[codes.int()].flatten(-2).unflatten(-1, (-1, GROUP))
    return (x * scale[..., None].float()).flatten(-2)


def load_rows(pool, slots, d, which):
    """Values [T, H, d] (fp32) of the tokens at `slots`."""
    blk, off = slots // BLOCK, slots % BLOCK
    lay = record_layout(d, pool.device)
    h = torch.arange(pool.shape[1], device=pool.device)[None, :, None]
    codes = pool[blk[:, None, None], h, lay[which][off][:, None, :]]
    two = torch.arange(2, device=pool.device)
    raw = pool[blk[:, None, None, None], h[..., None], lay[2 + which][off][:, None, :, None] + two]
    x = byte_values(pool.device)[codes.int()].flatten(-2).unflatten(-1, (-1, GROUP))
    return (x * raw.view(torch.bfloat16).float()).flatten(-2)


# ---- inputs -------------------------------------------------------------------

def _pool(gen, blocks, heads, d, std=0.5):
    """A pool whose pages hold quantised normal values: a bank of 256 pages,
    one drawn for each (block, head)."""
    bank = torch.empty(256, 1, record_bytes(d), dtype=torch.uint8, device="cuda")
    page = torch.arange(256, device="cuda").repeat_interleave(BLOCK)
    off = torch.arange(BLOCK, device="cuda").repeat(256)
    for which in (0, 1):
        x = torch.randn(256 * BLOCK, 1, d, generator=gen, device="cuda") * std
        store(bank, page, off, *quantise(x), which)
    pick = torch.randint(0, 256, (blocks * heads,), generator=gen, device="cuda")
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
    """Distinct slots of `tokens` tokens: runs of consecutive positions, each
    from an offset of its own, over shuffled blocks."""
    runs = -(-tokens // run)
    per = -(-run // BLOCK) + 1
    blocks = int(runs * per * 1.25) + 1
    perm = torch.randperm(blocks, generator=gen, device="cuda")
    start = torch.randint(0, BLOCK, (runs,), generator=gen, device="cuda")
    t = torch.arange(tokens, device="cuda")
    pos = start[t // run] + t % run
    return blocks, perm[(t // run) * per + pos // BLOCK] * BLOCK + pos % BLOCK, t % run


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    op = case["op"]
    s = dict(op=op, case=case)
    if op == "metadata":
        B, W, M = case["seqs"], case["width"], case["max_tokens"]
        std = torch.randn(2, B, generator=gen, device="cuda")
        cap = W * BLOCK
        ctx = (case["context_median"] * (0.8 * std[0]).exp()).round().clamp(1, cap // 2).int()
        fresh = torch.rand(B, generator=gen, device="cuda") < case["prompts"]
        new = (case["prompt_median"] * (0.8 * std[1]).exp()).round().clamp(1, cap // 2).int()
        nc = torch.where(fresh, 0, ctx)
        nn = torch.where(fresh, new, 1)
        room = M - (nn.cumsum(0) - nn)             # what does not fit the step stays idle
        nn = torch.minimum(nn, room.clamp(min=0))
        have, need = (nc + BLOCK - 1) // BLOCK, (nc + nn + BLOCK - 1) // BLOCK
        total = int(need.sum())
        blocks = int(total * 1.1) + 8
        perm = torch.randperm(blocks, generator=gen, device="cuda").int()
        col = torch.arange(W, device="cuda")[None, :]
        at = (have.cumsum(0) - have)[:, None] + col
        used = int(have.sum())
        tables = torch.where(col < have[:, None], perm[at.clamp(max=blocks - 1)], -1)
        free = torch.zeros(blocks, dtype=torch.int32, device="cuda")
        free[:blocks - used] = perm[used:]
        s.update(nc=nc.int(), nn=nn.int(), tables=tables.int().contiguous(), free=free,
                 num_free=torch.tensor([blocks - used], dtype=torch.int32, device="cuda"),
                 num_free_out=torch.zeros(1, dtype=torch.int32, device="cuda"),
                 token_seq=torch.empty(M, dtype=torch.int32, device="cuda"),
                 positions=torch.empty(M, dtype=torch.int32, device="cuda"),
                 slots=torch.empty(M, dtype=torch.int64, device="cuda"),
                 lens=torch.empty(B, dtype=torch.int32, device="cuda"),
                 totals=torch.empty(4, dtype=torch.int32, device="cuda"))
        return s
    d, H = case["head_dim"], case["kv_heads"]
    if op in ("write", "read"):
        blocks, slots, pos = _slots(gen, case["tokens"], case["run"])
        T = case["tokens"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s.update(pool=_pool(gen, blocks, H, d), slots=slots.contiguous(), pos=pos.int(),
                 k_out=torch.empty(T, H, d, dtype=dt, device="cuda"),
                 v_out=torch.empty(T, H, d, dtype=dt, device="cuda"))
        if op == "write":
            k, v = (torch.randn(T, H, d, generator=gen, device="cuda") * 0.5 for _ in range(2))
            if case["run"] == 1:      # decode tokens: positions anywhere
                s["pos"] = torch.randint(0, 8192, (T,), generator=gen, device="cuda").int()
            s.update(k=k.to(dt), v=v.to(dt))
        return s
    lens = _contexts(case, seed)
    B, G = case["seqs"], case["group"]
    W = max(1, -(-max(lens) // BLOCK))
    pages = [-(-c // BLOCK) for c in lens]
    blocks = int(sum(pages) * 1.05) + 1
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    need = torch.tensor(pages, device="cuda")
    perm = torch.randperm(blocks, generator=gen, device="cuda").int()
    col = torch.arange(W, device="cuda")[None, :]
    at = (need.cumsum(0) - need)[:, None] + col
    tables = torch.where(col < need[:, None], perm[at.clamp(max=blocks - 1)], -1).contiguous()
    dt = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    s.update(pool=_pool(gen, blocks, H, d), tables=tables, lens=cl, max_len=W * BLOCK,
             q=(torch.randn(B, H * G, d, generator=gen, device="cuda") * 0.5).to(torch.bfloat16),
             scale=d ** -0.5, out=torch.empty(B, H * G, d, dtype=dt, device="cuda"))
    # the split-K workspace a program keeps: per (sequence, query head) one slot
    # more than the partitions, each a maximum, a sum and a row of output
    part = -(-W * BLOCK // case["partition"]) + 1
    rows = B * H * G
    s["workspace"] = torch.empty(4 * rows * part * (d + 2) + 8 * rows + 4096, dtype=torch.uint8, device="cuda")
    return s


# ---- one pass -------------------------------------------------------------------

def _metadata_plain(s):
    nc, nn, W, M = s["nc"].long(), s["nn"].long(), s["tables"].shape[1], s["slots"].shape[0]
    B = nc.shape[0]
    have, need = (nc + BLOCK - 1) // BLOCK, (nc + nn + BLOCK - 1) // BLOCK
    grow = need - have
    cum = nn.cumsum(0)
    off = grow.cumsum(0) - grow
    col = torch.arange(W, device="cuda")[None, :]
    take = s["num_free"] - 1 - (off[:, None] + col - have[:, None])
    new = (col >= have[:, None]) & (col < need[:, None])
    s["tables"].copy_(torch.where(new, s["free"][take.clamp(0, s["free"].shape[0] - 1)], s["tables"]))
    t = torch.arange(M, device="cuda")
    live = t < cum[-1]
    seq = torch.searchsorted(cum, t, right=True).clamp(max=B - 1)
    pos = torch.where(live, nc[seq] + t - (cum - nn)[seq], -1)
    slot = s["tables"][seq, (pos // BLOCK).clamp(0, W - 1)].long() * BLOCK + pos % BLOCK
    s["token_seq"].copy_(torch.where(live, seq, 0))
    s["positions"].copy_(pos)
    s["slots"].copy_(torch.where(live, slot, -1))
    s["lens"].copy_(nc + nn)
    s["num_free_out"].copy_(s["num_free"] - grow.sum())
    s["totals"].copy_(torch.stack([cum[-1], (nc + nn).amax(), s["num_free"][0] - grow.sum(), cum[-1] * 0]))


def _rotate(x, pos, style, theta):
    """RoPE of x [T, H, d] in 64 bits."""
    x, d = x.double(), x.shape[-1]
    if style == "none":
        return x
    freq = theta ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device=x.device) / d)
    ang = pos.double()[:, None, None] * freq
    c, n = ang.cos(), ang.sin()
    a, b = (x[..., 0::2], x[..., 1::2]) if style == "gptj" else (x[..., :d // 2], x[..., d // 2:])
    y = (a * c - b * n, b * c + a * n)
    return torch.stack(y, -1).flatten(-2) if style == "gptj" else torch.cat(y, -1)


def _read_plain(s):
    for which, out in ((0, s["k_out"]), (1, s["v_out"])):
        out.copy_(load_rows(s["pool"], s["slots"], out.shape[-1], which))


def _write_plain(s):
    c = s["case"]
    blk, off = s["slots"] // BLOCK, s["slots"] % BLOCK
    k = _rotate(s["k"], s["pos"], c["rope"], c["theta"]).to(s["k"].dtype)
    store(s["pool"], blk, off, *quantise(k), 0)
    store(s["pool"], blk, off, *quantise(s["v"]), 1)


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
        if op == "metadata":
            pk.photon_build_step_metadata_device(
                s["nc"], s["nn"], s["tables"], s["free"], s["num_free"], s["token_seq"], s["positions"],
                s["slots"], s["lens"], s["totals"], num_free_out=s["num_free_out"])
        elif op == "decode":
            pk.photon_paged_attention_decode_fp4(s["q"], s["pool"], s["tables"], s["lens"], s["scale"], s["out"],
                                                 s["max_len"], c["partition"], s["workspace"])
        else:
            if op == "write":
                pk.photon_kv_cache_write_fp4(s["k"], s["v"], s["pos"], s["slots"], s["pool"], c["theta"], c["rope"])
            pk.photon_kv_cache_read_fp4(s["pool"], s["slots"], s["k_out"], s["v_out"])
    elif op == "metadata":
        _metadata_plain(s)
    elif op == "decode":
        _decode_plain(s)
    else:
        if op == "write":
            _write_plain(s)
        _read_plain(s)
    if op == "metadata":
        return [s["token_seq"], s["positions"], s["slots"], s["lens"], s["totals"], s["num_free_out"], s["tables"]]
    return [s["out"]] if op == "decode" else [s["k_out"], s["v_out"]]


def work(case):
    op = case["op"]
    if op == "metadata":
        B, M = case["seqs"], case["max_tokens"]
        # lengths in and out, three lists, and one table entry read per token or grown block
        return dict(bytes=12.0 * B + 16.0 * M + 4.0 * (B + M // BLOCK), flops=0.0)
    d, H = case["head_dim"], case["kv_heads"]
    token = H * record_bytes(d) / BLOCK            # 4-bit bytes of a token's K and V
    if op in ("write", "read"):
        T = case["tokens"]
        wide = 2 * H * d * (2 if case["dtype"] == "bf16" else 4)
        passes = 2 if op == "write" else 1         # written and read back
        return dict(bytes=T * (passes * (wide + token) + (12 if op == "write" else 8)), flops=0.0)
    lens = _contexts(case, 0)
    total, rows = sum(lens), case["seqs"] * H * case["group"]
    size = 2 if case["out"] == "bf16" else 4
    return dict(bytes=total * token + rows * d * (2 + size) + 4.0 * sum(-(-c // BLOCK) for c in lens),
                flops=4.0 * total * H * case["group"] * d)


# ---- the definition in 64 bits ------------------------------------------------------

def _values64(rec, d, which):
    """Values [16, d] (fp64) of one record's K or V, value by value from its bytes."""
    r = torch.arange(BLOCK, device=rec.device)[:, None]
    e = torch.arange(d, device=rec.device)[None, :]
    if which == 0:
        lane = (2 * (r // 4) + r % 2) * 4 + e % 64 // 16
        byte = e // 64 * 512 + lane * 16 + (r // 2 % 2) * 8 + e % 16 // 2
    else:
        byte = 8 * d + e // 64 * 512 + ((e % 64 // 8) * 4 + r // 4) * 16 + r % 4 * 4 + e % 8 // 2
    code = (rec[..., byte].long() >> (4 * (e % 2))) & 15
    at = 16 * d + e // 64 * 64 + r // 4 * 16 + which * 8 + r % 4 * 2
    bits = rec[..., at].int() | (rec[..., at + 1].int() << 8)
    scale = (bits << 16).view(torch.float32).double()
    ex, man = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(ex == 0, 0.5 * man, (1 + 0.5 * man) * torch.exp2((ex - 1).double()))
    return torch.where(code >= 8, -mag, mag) * scale


def exact(case, seed):
    if case["op"] == "metadata":      # whole numbers
        return None
    s, op = prepare(case, seed), case["op"]
    d, H = case["head_dim"], case["kv_heads"]
    if op == "decode":
        G = case["group"]
        out = torch.zeros(case["seqs"], H * G, d, dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["lens"].tolist()):
            if n:
                rec = s["pool"][s["tables"][b, :-(-n // BLOCK)].long()].transpose(0, 1)
                k, v = (_values64(rec, d, w).flatten(1, 2)[:, :n] for w in (0, 1))
                q = s["q"][b].double().view(H, G, d)
                out[b] = (torch.softmax(q @ k.mT * s["scale"], -1) @ v).view(H * G, d)
        return [out]
    if op == "read":
        blk, off = s["slots"] // BLOCK, s["slots"] % BLOCK
        rows = torch.arange(len(blk), device="cuda")
        step, got = 2048, ([], [])
        for t in range(0, len(blk), step):
            rec = s["pool"][blk[t:t + step]]
            for w in (0, 1):
                got[w].append(_values64(rec, d, w)[rows[:len(rec)], :, off[t:t + step]])
        return [torch.cat(g) for g in got]
    k = _rotate(s["k"], s["pos"], case["rope"], case["theta"]).to(s["k"].dtype)
    grid = torch.tensor(sorted({-m for m in MAGNITUDES} | set(MAGNITUDES)), dtype=torch.float64, device="cuda")
    even = torch.tensor([MAGNITUDES.index(abs(g)) % 2 == 0 for g in grid.tolist()], device="cuda")
    res = []
    for x in (k, s["v"]):
        g = x.double().unflatten(-1, (-1, GROUP))
        sc = (g.abs().amax(-1, keepdim=True).float() / 6).to(torch.bfloat16).double()
        y = (g / sc.clamp(min=1e-300)).clamp(-6, 6)
        hi = torch.searchsorted(grid, y.contiguous()).clamp(1, len(grid) - 1)
        up, down = grid[hi] - y, y - grid[hi - 1]
        hi = torch.where((down < up) | ((down == up) & even[hi - 1]), hi - 1, hi)
        res.append((grid[hi] * sc).flatten(-2))
    return res
