"""What the paged 4-bit KV cache operators are measured on.

Five operators that a serving step strings together:

* ``table``  build_page_table: block tables, slot maps and positions from request lengths;
* ``rope``   qk_norm_rope: per-head RMS norm of q and k with the position rotation;
* ``cache``  kv_write_q4 followed by kv_read_q4: rows into the 4-bit cache and back out of it;
* ``attn``   attn_decode_q4: one query token per request over the 4-bit paged cache.

``run`` computes each in elementary torch operations (``own`` false) or through the
framework's calls (``own`` true).  The state is the same for both: the 4-bit cache is held in
the framework's record format, which the plain form unpacks by itself.

Record format (one record = 16 tokens of one kv head, 18 d bytes; d = head_dim; G = d / 32
groups of 32 channels, each with one scale):
  K codes   at 0:    token r, t < 4, group w: 32-bit word at r d/2 + t d/8 + 4 w holding channels
                     32 w + 8 t + e, e < 8: code + 8 in the 4 bits at 16 (e % 2) + 4 (e / 2), the
                     word then rotated left by 3;
  V codes   at 8 d:  16-bit half (r % 2) of the 32-bit word at (r / 8) 4 d + (4 g + t) d/8 + 4 j,
                     t = (r % 8) / 2, g < 8, holding channels g d/8 + 4 j + i, i < 4: code + 8 in
                     the bits 4 i;
  K scales  at 16 d: bf16 [16 tokens][G];
  V scales  at 17 d: bf16 [G][16 tokens].
A value is code x scale.  The scale is max|x| / 7 cut to 5 significant bits, so that every
stored value is exactly a bf16 number.
"""
import math
import random

import torch

own = False

REC = 16                 # tokens per record
LOW, HIGH = 2.0 ** -100, 2.0 ** 120


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One decode step of a batch of 16: every request grows by a token (latency).
        dict(name="table step B16", op="table", B=16, page=64, old_max=131072, new_max=1, ragged=False, window=0),
        # The block tables of a few dozen ragged prompts admitted together, some of them
        # continuing; the slot map has one entry per prompt token.
        dict(name="table prompts B48", op="table", B=48, page=64, old_max=4096, new_max=32768, ragged=True, window=0),
        # The q and k of one decode step, Qwen3-4B-shaped heads (latency).
        dict(name="rope step N16", op="rope", N=16, Hq=32, Hkv=8, d=128, rot=128, norm=True, inter=False, start=131000),
        # The same layer over a whole prompt, read out of the packed q|k|v projection.
        dict(name="rope prompt N32768", op="rope", N=32768, Hq=32, Hkv=8, d=128, rot=128, norm=True, inter=False, start=0),
        # 64-channel heads, half of them rotated in neighbouring pairs, no norm, odd length.
        dict(name="rope d64 N5003", op="rope", N=5003, Hq=14, Hkv=2, d=64, rot=32, norm=False, inter=True, start=77),
        # One token per request into the cache and back (the append of a decode step).
        dict(name="cache append N16", op="cache", N=16, Hkv=8, d=128, page=64, ragged=True),
        # A prompt of 65536 tokens of one layer into the cache, and back out of it.
        dict(name="cache prompt N65536", op="cache", N=65536, Hkv=8, d=128, page=64, ragged=False),
        # Short single request (latency): the group of 4 query heads per kv head of both models.
        dict(name="attn B1 S4095", op="attn", B=1, S=4095, ragged=False, Hq=32, Hkv=8, d=128, page=64, sa=False),
        # A ragged batch of small 64-channel heads, small pages.
        dict(name="attn d64 B24 S9000", op="attn", B=24, S=9000, ragged=True, Hq=16, Hkv=2, d=64, page=16, sa=False),
        # A ragged batch of mid-length requests.
        dict(name="attn B16 S32768", op="attn", B=16, S=32768, ragged=True, Hq=32, Hkv=8, d=128, page=64, sa=False),
        # The long-context decode workload: 16 requests of 131072 tokens, an FA layer.
        dict(name="attn B16 S131072", op="attn", B=16, S=131072, ragged=False, Hq=32, Hkv=8, d=128, page=128, sa=False),
        # The same batch in an SA layer: the first block and the last 16 blocks of 128.
        dict(name="attn SA B16 S131072", op="attn", B=16, S=131072, ragged=False, Hq=32, Hkv=8, d=128, page=128, sa=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["table", "rope", "cache", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128, 48])
    if op == "table":
        B = _log(rng, 1, 512)
        return dict(op=op, B=B, page=page, old_max=_log(rng, 1, 16384),
                    new_max=rng.choice([1, _log(rng, 2, 130000 // B)]), ragged=rng.random() < 0.7,
                    window=rng.choice([0, 0, rng.randint(1, 24)]))
    if op == "rope":
        d = rng.choice([64, 128, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        return dict(op=op, N=_log(rng, 1, 30000), Hq=Hkv * rng.randint(1, 4 if Hkv == 8 else 8), Hkv=Hkv,
                    d=d, rot=rng.choice([d, d, d // 2]), norm=rng.random() < 0.7,
                    inter=rng.random() < 0.3, start=_log(rng, 1, 131072))
    if op == "cache":
        return dict(op=op, N=_log(rng, 1, 60000), Hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]),
                    page=page, ragged=rng.random() < 0.6)
    Hkv = rng.choice([1, 2, 4, 8])
    B = _log(rng, 1, 64)
    return dict(op=op, B=B, S=_log(rng, 1, min(131072, 1500000 // B)), ragged=rng.random() < 0.6,
                Hq=Hkv * rng.randint(1, 8), Hkv=Hkv, d=rng.choice([64, 128]), page=page,
                sa=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)


def _normal(shape, g, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _lengths(n, top, ragged, seed, low=1):
    """n request lengths: all `top`, or spread evenly over the logarithm up to `top` (with
    low = 0 every third of them empty), their order by the seed."""
    if not ragged:
        return [top] * n
    got = [0 if low == 0 and k % 3 == 1 else int(round(top ** ((k + 1) / n))) for k in range(n)]
    random.Random(seed).shuffle(got)
    return got


def _quantise(x):
    """Codes (float, -7..7) and scales of x [..., d] in groups of 32 channels."""
    g = x.float().unflatten(-1, (x.shape[-1] // 32, 32))
    a = g.abs().amax(-1)
    s = ((a / 7).view(torch.int32) & -0x80000).view(torch.float32)   # 5 significant bits
    s = torch.where(a < LOW, 0.0, s)
    n = torch.where(s[..., None] > 0, torch.round(g / s[..., None]), 0.0)
    bad = ~(a <= HIGH)
    return torch.where(bad[..., None], 0.0, n), torch.where(bad, math.nan, s)


def _pack(kn, ks, vn, vs):
    """Records [..., 18 d] uint8 from codes [..., 16, G, 32] and scales [..., 16, G]."""
    G = kn.shape[-2]
    d = 32 * G
    lead = kn.shape[:-3]
    at = torch.tensor([16 * (e % 2) + 4 * (e // 2) for e in range(8)], device=kn.device)
    u = (kn + 8).to(torch.int64).reshape(*lead, 16, G, 4, 8)
    w = (u << at).sum(-1)                                             # [..., 16, G, 4]
    w = ((w << 3) | (w >> 29)) & 0xFFFFFFFF
    kc = w.transpose(-1, -2).reshape(*lead, 16 * d // 8).to(torch.int32)
    u = (vn + 8).to(torch.int64).reshape(*lead, 2, 4, 2, 8, d // 32, 4)   # hi, t, parity, g, j, i
    h = (u << (4 * torch.arange(4, device=kn.device))).sum(-1)        # [..., hi, t, parity, g, j]
    w = h.select(-3, 0) | (h.select(-3, 1) << 16)                     # [..., hi, t, g, j]
    vc = w.transpose(-2, -3).reshape(*lead, 16 * d // 8).to(torch.int32)
    sk = ks.to(torch.bfloat16).reshape(*lead, 16 * G)
    sv = vs.to(torch.bfloat16).transpose(-1, -2).reshape(*lead, 16 * G)
    return torch.cat([x.contiguous().view(torch.uint8) for x in (kc, vc, sk, sv)], -1)


def _pool(pages, Hkv, page, d, g):
    """A cache of random rows, packed."""
    recs = pages * Hkv * (page // REC)
    out = torch.empty((recs, 18 * d), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (16 * d))
    for i in range(0, recs, step):
        m = min(step, recs - i)
        kn, ks = _quantise(_normal((m, 16, d), g))
        vn, vs = _quantise(_normal((m, 16, d), g))
        out[i:i + m] = _pack(kn, ks, vn, vs)
    return out.view(pages, Hkv, page // REC, 18 * d)


def _mask_of(case):
    """(sink blocks, window blocks, block) of an SA layer."""
    return 1, 16, 128


def _table_sizes(case, seed):
    page = case["page"]
    old = _lengths(case["B"], case["old_max"], True, seed, 0)
    new = [o + n for o, n in zip(old, _lengths(case["B"], case["new_max"], case["ragged"], seed + 1))]
    return page, old, new


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "table":
        page, old, new = _table_sizes(case, seed)
        B, sink, window = case["B"], (1 if case["window"] else 0), case["window"]
        cap = sink + window if window else 1 << 30
        width = -(-(case["old_max"] + case["new_max"]) // page) + 3
        total = sum(min(-(-n // page), cap) for n in new)
        ids = torch.randperm(total + 100, generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32)
        used = 0
        host = ids.cpu()
        for b in range(B):
            p = -(-old[b] // page)
            a = min(p, cap)
            mine = host[used:used + a]
            used += a
            if p:
                j = torch.arange(p)
                table[b, :p] = mine[torch.where(j < cap, j, sink + (j - sink) % max(window, 1))]
        room = sum(n - o for o, n in zip(old, new)) + (5 if case["ragged"] else 0)
        i32 = dict(dtype=torch.int32, device="cuda")
        return dict(op=op, page=page, sink=sink, window=window,
                    old=torch.tensor(old, **i32), new=torch.tensor(new, **i32), free=ids,
                    cursor=torch.tensor([used], **i32), cursor_out=torch.empty(1, **i32),
                    table=table.cuda(), slots=torch.empty(room, dtype=torch.int64, device="cuda"),
                    pos=torch.empty(room, **i32), cu=torch.empty(B + 1, **i32))
    if op == "rope":
        N, Hq, Hkv, d = case["N"], case["Hq"], case["Hkv"], case["d"]
        qkv = _normal((N, (Hq + 2 * Hkv) * d), g, 2.0)
        rot = case["rot"]
        inv = (1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
        w = [(1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16) if case["norm"] else None
             for _ in range(2)]
        pos = (case["start"] + torch.arange(N, device="cuda")).to(torch.int32)
        return dict(op=op, qkv=qkv, Hq=Hq, Hkv=Hkv, d=d, inv=inv, qw=w[0], kw=w[1], pos=pos, inter=case["inter"],
                    q_out=torch.empty((N, Hq, d), dtype=torch.bfloat16, device="cuda"),
                    k_out=torch.empty((N, Hkv, d), dtype=torch.bfloat16, device="cuda"))
    if op == "cache":
        N, Hkv, d, page = case["N"], case["Hkv"], case["d"], case["page"]
        qkv = _normal((N, 4 * Hkv * d), g)               # q|k|v with twice as many q channels
        pages = 2 * -(-N // page) + 70
        ids = torch.randperm(pages, generator=g, device="cuda")
        i = torch.arange(N, device="cuda")
        if not case["ragged"]:                            # one prompt from its first token
            slots = ids[i // page] * page + i % page
        elif N <= 64:                                     # one token for each request
            slots = ids[i] * page + torch.randint(0, page, (N,), generator=g, device="cuda")
        else:                                             # a prompt that continues inside a page
            slots = ids[(i + 7) // page] * page + (i + 7) % page
        shape = (N, Hkv, d)
        return dict(op=op, qkv=qkv, Hkv=Hkv, d=d, page=page, slots=slots, row=i,
                    pool=torch.zeros((pages, Hkv, page // REC, 18 * d), dtype=torch.uint8, device="cuda"),
                    k_out=torch.empty(shape, dtype=torch.bfloat16, device="cuda"),
                    v_out=torch.empty(shape, dtype=torch.bfloat16, device="cuda"))
    B, S, d, page = case["B"], case["S"], case["d"], case["page"]
    lens = _lengths(B, S, case["ragged"], seed)
    width = -(-S // page)
    need = [-(-n // page) for n in lens]
    pool = _pool(sum(need) + 3, case["Hkv"], page, d, g)
    ids = torch.randperm(pool.shape[0], generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
    q = _normal((B, case["Hq"], d), g)
    return dict(op=op, pool=pool, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), q=q,
                mode=torch.tensor([0 if case["sa"] else 1], dtype=torch.uint8, device="cuda"), sa=case["sa"],
                mask=_mask_of(case), o=torch.empty_like(q),
                lse=torch.empty((B, case["Hq"]), dtype=torch.float32, device="cuda"))


# ------------------------------------------------------------------ the framework's calls
_ctx = None


def _context():
    """The handle that a user's program makes once and keeps."""
    global _ctx
    if _ctx is None:
        from sparse_attention_flux_b200.flux import Context
        _ctx = Context(0)
    return _ctx


def _own(s):
    ctx = _context()
    if s["op"] == "table":
        ctx.build_page_table(s["old"], s["new"], s["free"], s["cursor"], s["cursor_out"], s["table"],
                             s["slots"], s["pos"], s["page"], sink_pages=s["sink"],
                             window_pages=s["window"], cu_new=s["cu"])
        return s["table"], s["slots"], s["pos"], s["cu"], s["cursor_out"]
    if s["op"] == "rope":
        N, Hq, Hkv, d = s["pos"].numel(), s["Hq"], s["Hkv"], s["d"]
        q = s["qkv"][:, :Hq * d].unflatten(1, (Hq, d))
        k = s["qkv"][:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
        ctx.qk_norm_rope(q, k, s["q_out"], s["k_out"], s["pos"], s["inv"], q_weight=s["qw"],
                         k_weight=s["kw"], eps=1e-6, interleaved=s["inter"])
        return s["q_out"], s["k_out"]
    if s["op"] == "cache":
        Hkv, d = s["Hkv"], s["d"]
        k = s["qkv"][:, 2 * Hkv * d:3 * Hkv * d].unflatten(1, (Hkv, d))
        v = s["qkv"][:, 3 * Hkv * d:].unflatten(1, (Hkv, d))
        ctx.kv_write_q4(k, v, s["slots"], s["pool"])
        ctx.kv_read_q4(s["pool"], s["slots"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    sink, window, block = s["mask"]
    ctx.attn_decode_q4(s["q"], s["pool"], s["table"], s["lens"], s["o"], 1 / math.sqrt(s["q"].shape[-1]),
                       layer_mode=s["mode"], layer=0, sink_blocks=sink, window_blocks=window, block=block,
                       lse=s["lse"])
    return s["o"], s["lse"]


# ------------------------------------------------------------------ the plain forms
def _plain_table(s):
    page, sink, window = s["page"], s["sink"], s["window"]
    cap = sink + window if window else 1 << 30
    old, new, table = s["old"].long(), s["new"].long(), s["table"]
    p0, p1 = (old + page - 1) // page, (new + page - 1) // page
    a0, a1 = p0.clamp(max=cap), p1.clamp(max=cap)
    end = (a1 - a0).cumsum(0)
    base = s["cursor"].long() + end - (a1 - a0)
    j = torch.arange(table.shape[1], device=table.device)[None]
    c = torch.where(j < cap, j, sink + (j - sink) % max(window, 1))
    fresh = s["free"][(base[:, None] + c - a0[:, None]).clamp(0, s["free"].numel() - 1)]
    kept = table.gather(1, c.expand(table.shape))
    table = torch.where((j >= p0[:, None]) & (j < p1[:, None]), torch.where(c >= a0[:, None], fresh, kept), table)
    cu = torch.cat([torch.zeros_like(end[:1]), (new - old).cumsum(0)])
    i = torch.arange(s["slots"].numel(), device=table.device)
    b = torch.bucketize(i, cu[1:].contiguous(), right=True).clamp(max=old.numel() - 1)
    pos = old[b] + i - cu[b]
    jt = (pos // page).clamp(max=table.shape[1] - 1)
    there = i < cu[-1]
    live = (jt < sink) | (jt >= p1[b] - window) if window else there
    slots = torch.where(there & live, table[b, jt].long() * page + pos % page, -1)
    return table, slots, torch.where(there, pos, 0).int(), cu.int(), s["cursor"] + end[-1:].int()


def _plain_rope(s):
    Hq, Hkv, d, inv = s["Hq"], s["Hkv"], s["d"], s["inv"]
    rot = 2 * inv.numel()
    angle = s["pos"].double()[:, None] * inv.double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = s["qkv"][:, :(Hq + Hkv) * d].float().unflatten(1, (Hq + Hkv, d))
    if s["qw"] is not None:
        w = torch.cat([s["qw"].float().expand(Hq, d), s["kw"].float().expand(Hkv, d)])
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if s["inter"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([a, b], -1).flatten(-2) if s["inter"] else torch.cat([a, b], -1)
    y = torch.cat([y, x[..., rot:]], -1).to(torch.bfloat16)
    return y[:, :Hq].contiguous(), y[:, Hq:].contiguous()


def _plain_cache(s):
    Hkv, d, N = s["Hkv"], s["d"], s["slots"].numel()
    x = s["qkv"][:, 2 * Hkv * d:].unflatten(1, (2, Hkv, d))
    n, sc = _quantise(x)
    y = (n * sc[..., None]).flatten(-2).to(torch.bfloat16)
    return y[:, 0].contiguous(), y[:, 1].contiguous()


def _unpack(rec, d):
    """fp32 K and V [..., 16, d] of records [..., 18 d]."""
    G, lead = d // 32, rec.shape[:-1]
    word = rec[..., :8 * d].contiguous().view(torch.int32).view(*lead, 16, 4, G).transpose(-1, -2)
    word = ((word >> 3) & 0x1FFFFFFF) | (word << 29)
    at = torch.tensor([16 * (e % 2) + 4 * (e // 2) for e in range(8)], dtype=torch.int32, device=rec.device)
    kn = ((word[..., None] >> at) & 15).reshape(*lead, 16, G, 32).float() - 8
    half = rec[..., 8 * d:16 * d].contiguous().view(torch.int16).view(*lead, 2, 8, 4, G, 2)   # hi, g, t, j, parity
    half = half.permute(*range(len(lead)), -5, -3, -1, -4, -2).int()                          # hi, t, parity, g, j
    vn = ((half[..., None] >> (4 * torch.arange(4, dtype=torch.int32, device=rec.device))) & 15)
    vn = vn.reshape(*lead, 16, G, 32).float() - 8
    ks = rec[..., 16 * d:17 * d].contiguous().view(torch.bfloat16).float().view(*lead, 16, G, 1)
    vs = rec[..., 17 * d:].contiguous().view(torch.bfloat16).float().view(*lead, G, 16).transpose(-1, -2)[..., None]
    return (kn * ks).flatten(-2), (vn * vs).flatten(-2)


def _plain_attn(s):
    q, lens, d = s["q"].float(), s["lens"].long(), s["q"].shape[-1]
    rec = s["pool"][s["table"].clamp(min=0).long()]                  # [B, pages, Hkv, records, 18 d]
    k, v = (x.transpose(1, 2).flatten(2, 4) for x in _unpack(rec, d))   # [B, Hkv, tokens, d]
    u = torch.arange(k.shape[2], device=q.device)[None]
    keep = u < lens[:, None]
    if s["sa"]:
        sink, window, block = s["mask"]
        keep = keep & ((u // block < sink) | (u // block >= ((lens + block - 1) // block)[:, None] - window))
    x = q.unflatten(1, (k.shape[1], -1)) @ k.transpose(-1, -2) * (1 / math.sqrt(d))
    x = x.masked_fill(~keep[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    o = (p @ v) / l
    return o.flatten(1, 2).to(torch.bfloat16), (m + torch.log(l)).flatten(1)


def run(state):
    if own:
        return _own(state)
    return {"table": _plain_table, "rope": _plain_rope, "cache": _plain_cache, "attn": _plain_attn}[state["op"]](state)


# ------------------------------------------------------------------ the work
def _live(n, sa, mask):
    if not sa:
        return n
    sink, window, block = mask
    first = max(0, -(-n // block) - window) * block
    return min(n, sink * block) + n - max(first, min(n, sink * block))


def work(case):
    op = case["op"]
    if op == "table":
        page, old, new = _table_sizes(case, 1)
        tokens, pages = sum(n - o for o, n in zip(old, new)), sum(-(-n // page) - -(-o // page) for o, n in zip(old, new))
        return {"bytes": 12 * tokens + 8 * pages + 12 * len(old) + 12, "flops": 0}
    if op == "rope":
        rows, d = case["N"] * (case["Hq"] + case["Hkv"]), case["d"]
        return {"bytes": 4 * rows * d + 4 * case["N"], "flops": rows * d * 7}
    if op == "cache":                                     # rows in, records out, records in, rows out
        rows, d = 2 * case["N"] * case["Hkv"], case["d"]
        return {"bytes": 2 * rows * (2 * d + d * 9 // 16) + 16 * case["N"], "flops": rows * d * 6}
    lens = _lengths(case["B"], case["S"], case["ragged"], 1)
    tokens = sum(_live(n, case["sa"], _mask_of(case)) for n in lens)
    d = case["d"]
    return {"bytes": tokens * case["Hkv"] * d * 9 // 8 + case["B"] * case["Hq"] * (4 * d + 4),
            "flops": 4 * tokens * case["Hq"] * d}


# ------------------------------------------------------------------ in 64 bits
def _exact_table(s):
    """Request by request, as a scheduler on the host would hand out pages."""
    page, sink, window = s["page"], s["sink"], s["window"]
    old, new, table, free = s["old"].tolist(), s["new"].tolist(), s["table"].cpu().numpy().copy(), s["free"].tolist()
    import numpy as np
    at, slots, pos, cu = int(s["cursor"]), [], [], [0]
    for b, (o, n) in enumerate(zip(old, new)):
        last = -(-n // page)
        for j in range(-(-o // page), last):
            if window and j >= sink + window:
                table[b, j] = table[b, j - window]
            else:
                table[b, j] = free[at]
                at += 1
        p = np.arange(o, n)
        j = p // page
        slot = table[b, j].astype(np.int64) * page + p % page
        slots.append(np.where((j < sink) | (j >= last - window), slot, -1) if window else slot)
        pos.append(p)
        cu.append(cu[-1] + n - o)
    rest = s["slots"].numel() - cu[-1]
    slots = np.concatenate(slots + [np.full(rest, -1)]).astype(np.int64)
    pos = np.concatenate(pos + [np.zeros(rest)]).astype(np.int32)
    return (torch.from_numpy(table), torch.from_numpy(slots), torch.from_numpy(pos),
            torch.tensor(cu, dtype=torch.int32), torch.tensor([at], dtype=torch.int32))


def _exact_rope(s):
    Hq, Hkv, d = s["Hq"], s["Hkv"], s["d"]
    half = s["inv"].numel()
    c = torch.arange(d, device="cuda")
    if s["inter"]:
        partner, index, first = c ^ 1, c // 2, c % 2 == 0
    else:
        partner, index, first = torch.where(c < half, c + half, c - half), c % half, c < half
    turned = c < 2 * half
    partner, index = torch.where(turned, partner, c), torch.where(turned, index, 0)
    angle = torch.where(turned, s["pos"].double()[:, None] * s["inv"].double()[index], 0.0)[:, None]
    out = []
    for x, w in ((s["qkv"][:, :Hq * d], s["qw"]), (s["qkv"][:, Hq * d:(Hq + Hkv) * d], s["kw"])):
        x = x.double().unflatten(1, (-1, d))
        if w is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + 1e-6) * w.double()
        other = x[..., partner]
        out.append(x * torch.cos(angle) + torch.where(turned, torch.where(first, -other, other), 0.0) * torch.sin(angle))
    return tuple(out)


def _exact_cache(s):
    """The grouped 4-bit rounding from its definition."""
    Hkv, d = s["Hkv"], s["d"]
    out = []
    for i in (2, 3):
        x = s["qkv"][:, i * Hkv * d:(i + 1) * Hkv * d].double().reshape(-1, 32)
        top = x.abs().max(1, keepdim=True).values
        mant, expo = torch.frexp(top / 7)
        scale = torch.ldexp(torch.floor(mant * 32) / 32, expo)
        n = torch.where(top >= LOW, torch.round(x / scale), 0.0)
        out.append((n * torch.where(top >= LOW, scale, 0.0)).view(-1, Hkv, d))
    return tuple(out)


def _exact_attn(s):
    """Token by token addresses into the records, then softmax in 64 bits."""
    q, d = s["q"].double(), s["q"].shape[-1]
    B, Hq, _ = q.shape
    Hkv, recs = s["pool"].shape[1], s["pool"].shape[2]
    page, flat = 16 * recs, s["pool"].view(-1, 18 * d)
    c = torch.arange(d, device="cuda")
    r = torch.arange(16, device="cuda")[:, None]
    bit = (16 * (c % 2) + 4 * (c % 8 // 2) + 3)                       # the rotated word's bits
    k_word = r * (d // 2) + c % 32 // 8 * (d // 8) + c // 32 * 4
    v_byte = 8 * d + r // 8 * 4 * d + (4 * (c // (d // 8)) + r % 8 // 2) * (d // 8) + c % (d // 8) // 4 * 4 + r % 2 * 2 + c % 4 // 2
    v_bit = 4 * (c % 2)
    outs, lses = [], []
    for b in range(B):
        n = int(s["lens"][b])
        u = torch.arange(n, device="cuda")
        if s["sa"]:
            sink, window, block = s["mask"]
            u = u[(u // block < sink) | (u // block >= -(-n // block) - window)]
        if not u.numel():
            outs.append(torch.zeros(Hq, d, dtype=torch.float64, device="cuda"))
            lses.append(torch.full((Hq,), -math.inf, dtype=torch.float64, device="cuda"))
            continue
        o, l = [], []
        for h in range(Hkv):
            rows = flat[(s["table"][b, u // page].long() * Hkv + h) * recs + u % page // 16]
            ru = u % 16
            code = 0
            for i in range(4):
                at = (bit + i) % 32
                byte = rows.gather(1, (k_word[ru] + at // 8))
                code = code + (((byte.int() >> (at % 8)) & 1) << i)
            sk = rows[:, 16 * d:17 * d].contiguous().view(torch.bfloat16).double().view(-1, 16, d // 32)
            k = (code - 8).double() * sk[torch.arange(len(u), device="cuda"), ru][:, c // 32]
            vcode = (rows.gather(1, v_byte[ru]).int() >> v_bit) & 15
            sv = rows[:, 17 * d:].contiguous().view(torch.bfloat16).double().view(-1, d // 32, 16)
            v = (vcode - 8).double() * sv[torch.arange(len(u), device="cuda"), :, ru][:, c // 32]
            x = q[b, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)] @ k.T / math.sqrt(d)
            l.append(torch.logsumexp(x, -1))
            o.append(torch.exp(x - l[-1][:, None]) @ v)
        outs.append(torch.cat(o))
        lses.append(torch.cat(l))
    return torch.stack(outs), torch.stack(lses)


def exact(case, seed):
    s = prepare(case, seed)
    return {"table": _exact_table, "rope": _exact_rope, "cache": _exact_cache, "attn": _exact_attn}[s["op"]](s)
