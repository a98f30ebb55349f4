"""Measured operators around the paged K/V cache's entries and scores.

append   queries and keys are normed per head (root mean square, with or without weights), rotated
         by a table of angles (halves or neighbours turning together, all of a head or its first
         dims, scaled for long contexts, positions of the sequence or given ones) and stored with
         the values in their sequences' pages, and each touched page's elementwise key bounds are
         brought up to date
attend   attention of every new token over its sequence's pages with scores that are capped by a
         tanh, biased by distance, or masked by documents packed into a sequence or by a prefix
         whose tokens see each other: one token per sequence, a few, or chunks
read     the entries of ragged ranges of positions come back out of the pages as rows in bf16

A cache is a pool of pages [page][kv head][slot][256] in bf16, or in E4M3 codes with one scale per
kv head for K and one for V; block i of a sequence holds its positions i * page_size onwards, in
the page that its row of the block table names.  Sliding layers attend to the last 512 positions,
their own among them.
"""
import functools
import math
import random

import torch

own = False

D = 256
WINDOW = 512
EPS = 1.0e-6
MAX_BATCH = 256
MAX_CONTEXT = 139264
# Angles: rotary dims, theta, which dims turn together, and the scaling for contexts beyond the trained ones.
TABLES = {
    "sliding": dict(rot=256, theta=1.0e4, pairs=False, scaling="none"),
    "full": dict(rot=64, theta=5.0e6, pairs=False, scaling="none"),
    "full linear": dict(rot=64, theta=5.0e6, pairs=False, scaling="linear", factor=4.0),
    "neighbours": dict(rot=128, theta=1.0e4, pairs=True, scaling="none"),
    "neighbours ramp": dict(rot=256, theta=1.0e4, pairs=True, scaling="ramp", factor=8.0, original=16384, slow=1.0, fast=32.0),
    "bands": dict(rot=256, theta=5.0e5, pairs=False, scaling="bands", factor=16.0, original=8192, slow=1.0, fast=4.0),
}


# ------------------------------------------------------------------- cases --

def _case(name, op, **kw):
    base = dict(name=name, op=op, layer="full", kv="bf16", q_heads=8, kv_heads=2, page=64, batch=1, ctx_lo=0, ctx_hi=0,
                tok_lo=1, tok_hi=1)
    if op == "append":
        base.update(table="full", weights=True, offset=0.0, fused=False, bounds=True, given=False)
    if op == "attend":
        base.update(sink=False, gate=False, softcap=0.0, spread=1.0, slopes=False, docs=0, prefix=0)
    base.update(kw)
    return base


def listed():
    return [
        # One token of each of 64 running sequences: a decode layer's entries, all latency.
        _case("norm append b64", "append", batch=64, ctx_lo=512, ctx_hi=32768),
        # Prompts of 8 sequences, ragged, q/k/v as parts of one projection's rows, E4M3 pages, neighbouring dims
        # turning together, scaled for a context eight times the trained one.
        _case("norm append 8 prompts e4m3", "append", table="neighbours ramp", kv="e4m3", q_heads=16, page=32, batch=8,
              ctx_lo=0, ctx_hi=4096, tok_lo=257, tok_hi=2047, fused=True, offset=1.0),
        # A packed prompt of 16384 tokens whose documents' positions start anew, without bounds.
        _case("norm append packed 16384", "append", table="bands", batch=1, tok_lo=16384, tok_hi=16384, bounds=False, given=True),
        # One sequence at 4096, scores capped: the latency of one decode layer.
        _case("capped b1 c4096", "attend", ctx_lo=4096, ctx_hi=4096, softcap=50.0, spread=8.0),
        # 64 running sequences, scores capped: bandwidth of the page reads.
        _case("capped b64", "attend", batch=64, ctx_lo=512, ctx_hi=32768, softcap=50.0, spread=8.0, sink=True),
        # Group 8, batch 256, E4M3 pages, a bias by distance and output gates.
        _case("distance b256 g8 e4m3", "attend", kv="e4m3", q_heads=16, page=128, batch=256, ctx_lo=512, ctx_hi=8192, slopes=True,
              gate=True),
        # Verification of 2 to 7 drafted tokens of 16 sequences, scores capped, 512-key windows.
        _case("capped tokens b16 sliding", "attend", layer="sliding", page=32, batch=16, ctx_lo=700, ctx_hi=8192, tok_lo=2,
              tok_hi=7, softcap=30.0, spread=6.0),
        # The last 4096 tokens of a 32768-token prompt, scores capped.
        _case("capped chunk 4096 of 32768", "attend", ctx_lo=28672, ctx_hi=28672, tok_lo=4096, tok_hi=4096, softcap=50.0,
              spread=8.0, sink=True),
        # Documents of some 60 to 2500 tokens packed into a prompt of 16384: each sees its own.
        _case("documents 16384", "attend", tok_lo=16384, tok_hi=16384, docs=1024),
        # Prompts of 3 sequences whose first part sees itself whole, bias by distance, group 8 over E4M3 pages.
        _case("prefix prompts g8 e4m3", "attend", kv="e4m3", q_heads=16, page=128, batch=3, tok_lo=1500, tok_hi=4000, slopes=True,
              prefix=1024),
        # 16 tokens of each of 32 sequences out of small pages: latency.
        _case("read b32", "read", page=16, batch=32, ctx_lo=0, ctx_hi=4096, tok_lo=1, tok_hi=16),
        # Four sequences of up to 32768 tokens out of E4M3 pages.
        _case("read 4 of 32768 e4m3", "read", kv="e4m3", batch=4, tok_lo=24576, tok_hi=32768),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "read"])
    group = rng.choice([1, 2, 4, 4, 8])
    kv_heads = rng.choice([1, 2, 2, 4])
    c = _case("", op, kv=rng.choice(["bf16", "bf16", "e4m3"]), kv_heads=kv_heads, q_heads=group * kv_heads,
              page=rng.choice([16, 32, 64, 128, 256]), batch=_log(rng, 1, 256))
    del c["name"]
    kind = rng.choice(["one", "few", "chunk"])
    if kind == "few":
        c["batch"] = min(c["batch"], 64)
        c["tok_hi"] = rng.randint(2, 9)
    if kind == "chunk":
        c["batch"] = min(c["batch"], 8)
        heads = c["batch"] * c["q_heads"]   # attend: at most 2^30 scores in all, as the largest listed case has
        most = 8192 // c["batch"] if op != "attend" else min(8192 // c["batch"], math.isqrt((1 << 29) // heads))
        c["tok_hi"] = _log(rng, 16, most)
    c["tok_lo"] = rng.randint(1, c["tok_hi"])
    if op == "append":
        c.update(table=rng.choice(sorted(TABLES)), weights=rng.random() < 0.8, offset=rng.choice([0.0, 1.0]),
                 fused=rng.random() < 0.5, bounds=rng.random() < 0.5, given=rng.random() < 0.3)
        c["ctx_hi"] = _log(rng, 1, 65536)
    elif op == "read":
        c["ctx_hi"] = _log(rng, 1, 65536)
    else:
        c.update(layer=rng.choice(["full", "full", "sliding"]), sink=rng.random() < 0.5, gate=rng.random() < 0.3,
                 softcap=rng.choice([0.0, 15.0, 30.0, 50.0]), spread=rng.choice([1.0, 4.0, 8.0]), slopes=rng.random() < 0.4)
        if kind == "chunk":
            c["docs"] = rng.choice([0, 0, 64, 512])
            c["prefix"] = 0 if c["docs"] else rng.choice([0, 0, _log(rng, 8, 2048)])
            room = (1 << 30) // (c["batch"] * c["q_heads"] * c["tok_hi"]) - c["tok_hi"]
            c["ctx_hi"] = _log(rng, 1, min(32768, room))
        else:
            keys = 1 << (21 if kind == "one" else 19)
            c["ctx_hi"] = _log(rng, 1, min(131072 if kind == "one" else 32768, keys // (c["batch"] * kv_heads)))
        if not (c["softcap"] or c["slopes"] or c["docs"] or c["prefix"]):
            c["softcap"] = 30.0
    c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
    return c


def _lengths(c):
    """(previous tokens, new tokens) of every sequence of a case."""
    rng = random.Random(1000 * c["batch"] + c["ctx_hi"] + 7 * c["tok_hi"])
    return ([rng.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["batch"])],
            [rng.randint(c["tok_lo"], c["tok_hi"]) for _ in range(c["batch"])])


def _documents(c):
    """First position of the document of every new token, sequence after sequence: documents of docs / 16 to 2.4 docs
    tokens, the first of which may have begun before."""
    rng = random.Random(31 * c["docs"] + c["tok_hi"])
    out = []
    for x, n in zip(*_lengths(c)):
        start = rng.randint(max(0, x - c["docs"]), x)
        row = []
        while len(row) < n:
            end = x + len(row) + rng.randint(max(1, c["docs"] // 16), max(1, 12 * c["docs"] // 5))
            while len(row) < n and x + len(row) < end:
                row.append(start)
            start = end
        out += row
    return out


def _prefixes(c):
    """Length of each sequence's prefix: up to twice the case's, some without."""
    rng = random.Random(17 * c["prefix"] + c["batch"])
    return [rng.choice([0, 1, 1, 1]) * rng.randint(1, 2 * c["prefix"]) for _ in range(c["batch"])]


def _spans(c):
    """[first, last] visible position of every new token (attend)."""
    docs = _documents(c) if c["docs"] else None
    prefix = _prefixes(c) if c["prefix"] else [0] * c["batch"]
    out = []
    for (x, n), pre in zip(zip(*_lengths(c)), prefix):
        for p in range(x, x + n):
            lo = max(0, p - WINDOW + 1) if c["layer"] == "sliding" else 0
            if docs:
                lo = max(lo, docs[len(out)])
            out.append((lo, max(p, min(pre, x + n) - 1) if p < pre else p))
    return out


def work(c):
    c = dict(_case("", c["op"]), **c)
    ctx, tok = _lengths(c)
    e = 1 if c["kv"] == "e4m3" else 2
    rows, Hq, Hkv, ps = sum(tok), c["q_heads"], c["kv_heads"], c["page"]
    touched = sum(-(-(x + n) // ps) - x // ps for x, n in zip(ctx, tok))
    tables = 4 * (2 * c["batch"] + 1 + touched)
    if c["op"] == "append":
        rot = TABLES[c["table"]]["rot"]
        nbytes = rows * D * (4 * Hq + 4 * Hkv + 2 * e * Hkv) + tables + rows * rot * 4 + (4 * rows if c["given"] else 0)
        if c["bounds"]:
            reused = sum(x % ps != 0 for x in ctx)   # pages whose bounds are read before they are written
            nbytes += (touched + reused) * Hkv * 2 * D * 2
        return {"bytes": nbytes, "flops": rows * (Hq + Hkv) * (4 * D + 3 * rot)}
    if c["op"] == "read":
        return {"bytes": rows * Hkv * D * 2 * (e + 2) + tables, "flops": rows * Hkv * D * 2 if e == 1 else 0}
    spans = _spans(c)
    keys, r = 0, 0
    for n in tok:   # each read once
        keys += max(hi for _, hi in spans[r: r + n]) + 1 - min(lo for lo, _ in spans[r: r + n])
        r += n
    pairs = sum(hi - lo + 1 for lo, hi in spans)
    nbytes = keys * Hkv * D * 2 * e + rows * Hq * (4 * D + 4 + (4 if c["gate"] else 0)) + 4 * (rows if c["docs"] else 0)
    return {"bytes": nbytes + 4 * sum(-(-(x + n) // ps) for x, n in zip(ctx, tok)), "flops": pairs * Hq * D * 4}


# ------------------------------------------------------------------ inputs --

def prepare(case, seed):
    c = dict(_case("", case["op"]), **case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    Hq, Hkv, ps, B, op = c["q_heads"], c["kv_heads"], c["page"], c["batch"], c["op"]
    ctx, tok = _lengths(c)
    rows, nblk = sum(tok), -(-max(x + n for x, n in zip(ctx, tok)) // ps)
    off = [0]
    for n in tok:
        off.append(off[-1] + n)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    randn = lambda *shape: torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)  # noqa: E731

    # Which blocks of each sequence hold a page: those that the call touches; the others' entries name a page that no
    # call reads.
    lo, hi = [x // ps for x in ctx], [-(-(x + n) // ps) for x, n in zip(ctx, tok)]
    if op == "attend":
        spans = _spans(c)
        lo = [min(s[0] for s in spans[a: b]) // ps for a, b in zip(off, off[1:])]
    pool = sum(h - w for w, h in zip(lo, hi)) + 3
    order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    blk = torch.arange(nblk, device=dev).unsqueeze(0)
    lo_t, hi_t = torch.tensor(lo, device=dev).unsqueeze(1), torch.tensor(hi, device=dev).unsqueeze(1)
    start = torch.tensor([0] + [h - w for w, h in zip(lo, hi)], device=dev).cumsum(0)[:-1].unsqueeze(1)
    inside = (blk >= lo_t) & (blk < hi_t)
    table = order[torch.where(inside, start + blk - lo_t, torch.full_like(blk, pool - 1))].contiguous()

    s = {"case": c, "table": table, "nblk": nblk, "first_block": min(lo), "rows": rows, "max_tokens": max(tok),
         "max_context": max(ctx), "context": ints(ctx), "offsets": ints(off), "k_scale": None, "v_scale": None}
    s["seq"] = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(tok, device=dev))   # sequence of each row
    s["tok"] = torch.arange(rows, device=dev) - s["offsets"][s["seq"]].long()   # its number among the new tokens
    s["k"], s["v"] = randn(pool, Hkv, ps, D), randn(pool, Hkv, ps, D)
    if c["kv"] == "e4m3":
        for n in ("k", "v"):
            scale = (3 + 3 * torch.rand(Hkv, generator=g, device=dev)) / 448
            s[n + "_scale"] = scale
            s[n] = (s[n] / scale.view(1, -1, 1, 1).to(torch.bfloat16)).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
    if op == "append":
        q, k, v = randn(rows, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], dim=1)
        s["new"] = (q, k, v) if c["fused"] else (q.contiguous(), k.contiguous(), v.contiguous())
        s["q_rot"] = torch.empty(rows, Hq, D, dtype=torch.bfloat16, device=dev)
        for n in ("q_weight", "k_weight"):
            s[n] = None if not c["weights"] else ((1 - c["offset"]) + 0.25 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16)
        s["positions"] = None
        if c["given"]:   # documents whose positions start anew
            p = [t % 1777 for n in tok for t in range(n)]
            s["positions"] = ints(p)
        s["bounds"] = None
        if c["bounds"]:   # of the keys that the pages hold so far (an append into a fresh page starts anew)
            used = torch.zeros(pool, dtype=torch.int64, device=dev)
            held = (s["context"].long().unsqueeze(1) - blk * ps).clamp(0, ps)
            used[table.long()[inside]] = held[inside]
            dead = (torch.arange(ps, device=dev) >= used.unsqueeze(1)).view(pool, 1, ps, 1)
            x = s["k"].to(torch.bfloat16)
            s["bounds"] = torch.stack([x.masked_fill(dead, math.inf).amin(2), x.masked_fill(dead, -math.inf).amax(2)], 2).contiguous()
    elif op == "attend":
        s["q"] = randn(rows, Hq, D) * c["spread"]
        s["sink"] = torch.randn(Hq, generator=g, device=dev) if c["sink"] else None
        s["gate"] = torch.randn(rows, Hq, generator=g, device=dev) if c["gate"] else None
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=dev) / Hq) if c["slopes"] else None
        s["first"] = ints(_documents(c)) if c["docs"] else None
        s["last"] = ints([x for _, x in spans]) if c["prefix"] else None
        s["out"] = torch.empty(rows, Hq, D, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty(rows, Hq, dtype=torch.float32, device=dev)
    else:
        s["rows_k"], s["rows_v"] = (torch.empty(rows, Hkv, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    return s


# ------------------------------------------------------------- plain forms --

def _frequencies(t, dev):
    """Turn per position of each pair, in 64 bits, and the factor on cosines and sines."""
    rot = t["rot"]
    f = t["theta"] ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
    if t["scaling"] == "linear":
        return f / t["factor"], 1.0
    if t["scaling"] == "ramp":
        # Pairs that turn at least `fast` times over the trained context keep their speed, those that turn `slow` times
        # or less are slowed by the factor, in between by a ramp over the pairs' numbers.
        def number(turns):
            return rot * math.log(t["original"] / (turns * 2 * math.pi)) / (2 * math.log(t["theta"]))
        lo, hi = max(math.floor(number(t["fast"])), 0), min(math.ceil(number(t["slow"])), rot - 1)
        ramp = ((torch.arange(rot // 2, device=dev, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / t["factor"] * ramp, 0.1 * math.log(t["factor"]) + 1
    if t["scaling"] == "bands":
        # The same by a ramp over the number of turns itself.
        turns = t["original"] * f / (2 * math.pi)
        keep = ((turns - t["slow"]) / (t["fast"] - t["slow"])).clamp(0, 1)
        return f * keep + f / t["factor"] * (1 - keep), 1.0
    return f, 1.0


def _norm(x, weight, offset):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return y if weight is None else y * (weight.float() + offset)


def _rotate(x, pos, t):
    """Rotation of x [rows, heads, 256] by its row's position; the cosines and sines have 32 bits."""
    rot = t["rot"]
    f, m = _frequencies(t, x.device)
    a = pos.double().unsqueeze(1) * f
    cos, sin = ((h(a) * m).float().unsqueeze(1) for h in (torch.cos, torch.sin))
    if t["pairs"]:
        x1, x2 = x[..., :rot:2], x[..., 1:rot:2]
        y = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], dim=-1).flatten(-2)
    else:
        x1, x2 = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _place(s):
    """Page and slot of every row's entry."""
    ps = s["case"]["page"]
    pos = s["context"].long()[s["seq"]] + s["tok"]
    return pos, s["table"].long()[s["seq"], pos // ps], pos % ps


def _bytes(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _append(s):
    c = s["case"]
    q, k, v = s["new"]
    t = TABLES[c["table"]]
    pos, page, slot = _place(s)
    turn = pos if s["positions"] is None else s["positions"].long()
    s["q_rot"].copy_(_rotate(_norm(q, s["q_weight"], c["offset"]), turn, t))
    k = _rotate(_norm(k, s["k_weight"], c["offset"]), turn, t)
    if c["kv"] == "e4m3":
        k, v = ((x.float() / sc.view(1, -1, 1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
                for x, sc in ((k, s["k_scale"]), (v, s["v_scale"])))
    else:
        k = k.to(torch.bfloat16)
    _bytes(s["k"])[page, :, slot] = _bytes(k)
    _bytes(s["v"])[page, :, slot] = _bytes(v)
    out = {"q": s["q_rot"], "k": s["k"], "v": s["v"]}
    if s["bounds"] is not None:
        # A page whose first slot is written now starts anew; the others keep what they held.
        fresh = torch.zeros(s["k"].shape[0], device=q.device).index_reduce_(0, page, (slot == 0).float(), "amax").view(-1, 1, 1) > 0
        k = k.float()
        lo = torch.where(fresh, math.inf, s["bounds"][:, :, 0].float()).index_reduce_(0, page, k, "amin")
        hi = torch.where(fresh, -math.inf, s["bounds"][:, :, 1].float()).index_reduce_(0, page, k, "amax")
        s["bounds"].copy_(torch.stack([lo, hi], dim=2))
        out["bounds"] = s["bounds"]
    return out


def _read(s):
    _, page, slot = _place(s)
    for n in ("k", "v"):
        x = _bytes(s[n])[page, :, slot].view(s[n].dtype).float()
        s["rows_" + n].copy_(x if s[n + "_scale"] is None else x * s[n + "_scale"].view(1, -1, 1))
    return {"k": s["rows_k"], "v": s["rows_v"]}


def _values(t, scale, pages):
    """Slots [batch, kv head, n, slot, 256] of the pages [batch, kv head, n], in 32 bits."""
    head = torch.arange(t.shape[1], device=t.device).view(1, -1, 1)
    x = _bytes(t)[pages, head].view(t.dtype).float()
    return x if scale is None else x * scale.view(1, -1, 1, 1, 1)


def _attend(s):
    c = s["case"]
    B, N, Hkv, ps, nblk = c["batch"], s["max_tokens"], c["kv_heads"], c["page"], s["nblk"]
    G = c["q_heads"] // Hkv
    dev = s["q"].device
    # The blocks that a sequence's tokens see: all from the call's first on, or those from its first token's window on.
    first, n = torch.full((B, 1), s["first_block"], device=dev, dtype=torch.long), nblk - s["first_block"]
    if c["layer"] == "sliding":
        first = (s["context"].long() - WINDOW + 1).clamp(min=0).unsqueeze(1) // ps
        n = min(nblk, (WINDOW + N - 2) // ps + 2)
    blk = first + torch.arange(n, device=dev)
    key = (blk.unsqueeze(-1) * ps + torch.arange(ps, device=dev)).flatten(1)               # [B, keys]: their positions
    pages = s["table"].long().gather(1, blk.clamp(max=nblk - 1)).unsqueeze(1).expand(B, Hkv, n)
    k, v = (_values(s[n], s[n + "_scale"], pages).flatten(2, 3) for n in ("k", "v"))       # [B, Hkv, keys, D]
    # Queries padded to the longest sequence: [B, Hkv, N * G, D].
    t = torch.arange(N, device=dev)
    at = (s["offsets"][:-1].long().unsqueeze(1) + t).clamp(max=s["rows"] - 1)
    q = s["q"].float()[at].view(B, N, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, N * G, D)
    pos = s["context"].long().unsqueeze(1) + t                                             # [B, N]
    lo = pos - WINDOW + 1 if c["layer"] == "sliding" else torch.zeros_like(pos)
    if s["first"] is not None:
        lo = torch.maximum(lo, s["first"].long()[at])
    hi = pos if s["last"] is None else s["last"].long()[at]
    seen = (key.unsqueeze(1) <= hi.unsqueeze(-1)) & (key.unsqueeze(1) >= lo.unsqueeze(-1))   # [B, N, keys]
    score = (q @ k.transpose(-1, -2)).mul_(1 / 16).view(B, Hkv, N, G, -1)
    if c["softcap"]:
        score = score.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    if s["slopes"] is not None:
        far = (key.unsqueeze(1) - pos.unsqueeze(-1)).abs().float().view(B, 1, N, 1, -1)
        score = score.sub_(far * s["slopes"].view(1, Hkv, 1, G, 1))
    score = score.masked_fill_(~seen.view(B, 1, N, 1, -1), -math.inf).view(B, Hkv, N * G, -1)
    m = score.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(score - m)
    total = p.sum(-1)
    out = (p @ v) / total.unsqueeze(-1)
    lse = m.squeeze(-1) + torch.log(total)
    # [B, kv head, token * group, ..] -> [B, token, q head, ..] -> rows
    lse = lse.view(B, Hkv, N, G).transpose(1, 2).flatten(2)[s["seq"], s["tok"]]
    out = out.view(B, Hkv, N, G, D).transpose(1, 2).flatten(2, 3)[s["seq"], s["tok"]]
    if s["sink"] is not None:
        out = out * torch.sigmoid(lse - s["sink"]).unsqueeze(-1)
    if s["gate"] is not None:
        out = out * torch.sigmoid(s["gate"]).unsqueeze(-1)
    return {"out": out.to(torch.bfloat16), "lse": lse}


# ------------------------------------------------------ the framework's way --

@functools.lru_cache(maxsize=None)
def _context(q_heads, kv_heads, kv):
    """The context that a serving program keeps for its model: one sliding and one full layer here."""
    import full_gqa_decode_gb300 as hd
    return hd.hybrid_decode_init(hd.Config(layer_types=[hd.HD_SLIDING, hd.HD_FULL], num_q_heads=q_heads, num_kv_heads=kv_heads,
                                           sliding_window=WINDOW, max_batch=MAX_BATCH, max_context=MAX_CONTEXT,
                                           kv_dtype=hd.HD_KV_FP8_E4M3 if kv == "e4m3" else hd.HD_KV_BF16))


@functools.lru_cache(maxsize=None)
def _angles(name):
    """The table of angles that a serving program keeps for its model."""
    import full_gqa_decode_gb300 as hd
    t = TABLES[name]
    kw = dict(linear=dict(factor=t.get("factor")),
              ramp=dict(factor=t.get("factor"), original_context=t.get("original"), slow=t.get("slow"), fast=t.get("fast")),
              bands=dict(factor=t.get("factor"), original_context=t.get("original"), slow=t.get("slow"), fast=t.get("fast")),
              none={})[t["scaling"]]
    kind = dict(none=hd.HD_ROPE_PLAIN, linear=hd.HD_ROPE_LINEAR, ramp=hd.HD_ROPE_RAMP, bands=hd.HD_ROPE_BANDS)[t["scaling"]]
    return hd.rope_table(t["rot"], MAX_CONTEXT + 1, theta=t["theta"], scaling=kind,
                         layout=hd.HD_ROPE_NEIGHBOURS if t["pairs"] else hd.HD_ROPE_HALVES, **kw)


def _plan(s):
    """Descriptors of the batch, the cache and the scores, made once for a step's tensors."""
    import full_gqa_decode_gb300 as hd
    c = s["case"]
    offsets = None if c["tok_hi"] == 1 else s["offsets"]
    rule = None
    if c["op"] == "append":
        rule = _angles(c["table"])
    elif c["op"] == "attend":
        rule = hd.scoring(softcap=c["softcap"], slopes=s["slopes"], first=s["first"], last=s["last"])
    return (hd, _context(c["q_heads"], c["kv_heads"], c["kv"]), int(c["layer"] == "full"),
            hd.paged_batch(s["table"], s["context"], offsets, num_tokens=s["rows"], max_tokens=s["max_tokens"],
                           max_context=s["max_context"]),
            hd.paged_cache(s["k"], s["v"], s["k_scale"], s["v_scale"], bounds=s.get("bounds")), rule)


def _own(s):
    if "plan" not in s:
        s["plan"] = _plan(s)
    hd, ctx, layer, batch, cache, rule = s["plan"]
    c = s["case"]
    if c["op"] == "append":
        hd.norm_rope_append_paged(ctx, layer, batch, *s["new"], s["q_rot"], cache, rope=rule, q_weight=s["q_weight"],
                                  k_weight=s["k_weight"], eps=EPS, weight_offset=c["offset"], positions=s["positions"])
        out = {"q": s["q_rot"], "k": s["k"], "v": s["v"]}
        return out if s["bounds"] is None else dict(out, bounds=s["bounds"])
    if c["op"] == "read":
        hd.read_paged(ctx, batch, cache, s["rows_k"], s["rows_v"])
        return {"k": s["rows_k"], "v": s["rows_v"]}
    hd.attn_paged_scored(ctx, layer, batch, rule, s["q"], cache, s["sink"], s["out"], s["lse"], gate=s["gate"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"append": _append, "attend": _attend, "read": _read}[state["case"]["op"]](state)


# ------------------------------------------------------- 64-bit definitions --

def _exact_turns(t, dev):
    """exp(i turn) per position as a function of positions: pair j turns by its frequency, from the definitions."""
    rot, j = t["rot"], torch.arange(t["rot"] // 2, device=dev, dtype=torch.float64)
    f = torch.exp(-2 * j / rot * math.log(t["theta"]))
    size = 1.0
    if t["scaling"] == "linear":
        f = f / t["factor"]
    elif t["scaling"] != "none":
        if t["scaling"] == "ramp":
            edge = [rot / 2 * (math.log(t["original"] / (2 * math.pi)) - math.log(n)) / math.log(t["theta"]) for n in (t["fast"], t["slow"])]
            lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rot - 1)
            slowed = torch.clip((j - lo) / max(hi - lo, 1e-3), 0, 1)
            size = 1 + math.log(t["factor"]) / 10
        else:
            slowed = torch.clip((t["fast"] - t["original"] * f / math.tau) / (t["fast"] - t["slow"]), 0, 1)
        f = f * (1 + slowed * (1 / t["factor"] - 1))
    return lambda p: torch.polar(torch.full((), size, device=dev, dtype=torch.float64), p.double().unsqueeze(-1) * f)


def _exact_append(s):
    c = s["case"]
    t = TABLES[c["table"]]
    rot, ps = t["rot"], c["page"]
    pos = torch.cat([torch.arange(x, x + n, device=s["k"].device) for x, n in zip(*_lengths(c))])
    turn = _exact_turns(t, pos.device)(pos if s["positions"] is None else s["positions"]).unsqueeze(1)
    new = []
    for x, w in zip(s["new"][:2], (s["q_weight"], s["k_weight"])):
        x = x.double()
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS)
        if w is not None:
            x = x * (w.double() + c["offset"])
        even, odd = (slice(0, rot, 2), slice(1, rot, 2)) if t["pairs"] else (slice(0, rot // 2), slice(rot // 2, rot))
        z = torch.complex(x[..., even].contiguous(), x[..., odd].contiguous()) * turn
        x[..., even], x[..., odd] = z.real, z.imag
        new.append(x)
    q, k = new
    v = s["new"][2].double()
    pages = [s["k"].double(), s["v"].double()]
    bounds = None if s["bounds"] is None else s["bounds"].double()
    for i, n in ((0, "k"), (1, "v")):
        x = (k, v)[i]
        if c["kv"] == "e4m3":
            x = (x / s[n + "_scale"].double().view(1, -1, 1)).clamp(-448, 448)
        r = 0
        for b, (p0, m) in enumerate(zip(*_lengths(c))):
            for blk in range(p0 // ps, (p0 + m - 1) // ps + 1):
                a, e = max(p0, blk * ps), min(p0 + m, blk * ps + ps)
                page, part = int(s["table"][b, blk]), x[r + a - p0: r + e - p0].transpose(0, 1)
                pages[i][page, :, a - blk * ps: e - blk * ps] = part
                if i == 0 and bounds is not None:
                    old = bounds[page] if a > blk * ps else None
                    lo, hi = part.amin(1), part.amax(1)
                    bounds[page, :, 0] = lo if old is None else torch.minimum(old[:, 0], lo)
                    bounds[page, :, 1] = hi if old is None else torch.maximum(old[:, 1], hi)
            r += m
    out = {"q": q, "k": pages[0], "v": pages[1]}
    if bounds is not None:   # E4M3: the minima and maxima of rounded codes are the plain form's to say
        out["bounds"] = bounds if c["kv"] == "bf16" else None
    return out


def _exact_read(s):
    c = s["case"]
    ps, out = c["page"], {"k": [], "v": []}
    for n in ("k", "v"):
        scale = 1.0 if s[n + "_scale"] is None else s[n + "_scale"].double().view(-1, 1, 1)
        for b, (x, m) in enumerate(zip(*_lengths(c))):
            pages = s["table"][b, x // ps: -(-(x + m) // ps)].long()
            e = (_bytes(s[n])[pages].view(s[n].dtype).double() * scale).transpose(1, 2).flatten(0, 1)
            out[n].append(e[x % ps: x % ps + m])
    return {n: torch.cat(x) for n, x in out.items()}


def _exact_attend(s):
    c = s["case"]
    ps, Hkv = c["page"], c["kv_heads"]
    G = c["q_heads"] // Hkv
    dev = s["q"].device
    out = torch.empty(s["rows"], c["q_heads"], D, dtype=torch.float64, device=dev)
    lse = torch.empty(s["rows"], c["q_heads"], dtype=torch.float64, device=dev)
    spans = torch.tensor(_spans(c), device=dev)
    r0 = 0
    for b, (x, n) in enumerate(zip(*_lengths(c))):
        for t0 in range(0, n, 512):
            rows = slice(r0 + t0, r0 + min(n, t0 + 512))
            lo, hi = spans[rows, 0], spans[rows, 1]
            at0, at1 = int(lo.min()) // ps, int(hi.max()) // ps + 1
            at = torch.arange(at0 * ps, at1 * ps, device=dev)
            pages = s["table"][b, at0: at1].long()
            ok = (at >= lo.unsqueeze(1)) & (at <= hi.unsqueeze(1))
            p = torch.arange(x + t0, x + min(n, t0 + 512), device=dev)
            for h in range(Hkv):
                key, val = (_bytes(s[m])[pages, h].view(s[m].dtype).flatten(0, 1).double() *
                            (1.0 if s[m + "_scale"] is None else float(s[m + "_scale"][h])) for m in ("k", "v"))
                hs = slice(h * G, h * G + G)
                y = torch.einsum("thd,nd->thn", s["q"][rows, hs].double(), key) / 16
                if c["softcap"]:
                    e = torch.exp(-2 * y.abs() / c["softcap"])
                    y = torch.sign(y) * c["softcap"] * (1 - e) / (1 + e)
                if s["slopes"] is not None:
                    y = y - (at - p.unsqueeze(1)).abs().unsqueeze(1) * s["slopes"][hs].double().unsqueeze(1)
                y = y.masked_fill(~ok.unsqueeze(1), -math.inf)
                lse[rows, hs] = torch.logsumexp(y, -1)
                out[rows, hs] = torch.einsum("thn,nd->thd", torch.exp(y - lse[rows, hs].unsqueeze(-1)), val)
        r0 += n
    if s["sink"] is not None:
        out /= 1 + torch.exp(s["sink"].double() - lse).unsqueeze(-1)
    if s["gate"] is not None:
        out /= 1 + torch.exp(-s["gate"].double()).unsqueeze(-1)
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "read": _exact_read}[s["case"]["op"]](s)
