"""Measured operators of the paged K/V cache.

Three operators that a serving program calls one after the other in each layer:

append   new keys (rotated by their position) and values go into the pages of their
         sequences, the queries are rotated, and each touched page's elementwise key
         bounds are brought up to date
attend   attention of every new token over its sequence's pages: one token per sequence
         (decode), a few (verification of drafted tokens), or chunks of a prompt
select   for every new token, the pages with the largest bound on its scores are chosen,
         and it attends to those alone

A cache is a pool of pages [page][kv head][slot][256] in bf16, or in E4M3 codes with one
scale per kv head for K and one for V; block i of a sequence holds its positions
i * page_size onwards, in the page that its row of the block table names.  Sliding layers
attend to the last 512 positions, their own among them.
"""
import functools
import math
import random

import torch

own = False

D = 256
WINDOW = 512
ROPE = {"sliding": (256, 1.0e4), "full": (64, 5.0e6)}  # layer type -> (rotary dims, theta)
MAX_BATCH = 256
MAX_CONTEXT = 139264


# ------------------------------------------------------------------- cases --

def _case(name, op, **kw):
    base = dict(name=name, op=op, layer="full", kv="bf16", q_heads=8, kv_heads=2, page=64, batch=1, ctx_lo=0, ctx_hi=0,
                tok_lo=1, tok_hi=1, sink=False, gate=False, fused=False, pages=0)
    base.update(kw)
    return base


def listed():
    return [
        # One token of each of 64 running sequences of a full layer: the smallest append, all latency.
        _case("append b64", "append", batch=64, ctx_lo=512, ctx_hi=32768),
        # Prompts of 8 sequences, ragged, q/k/v as parts of one projection's rows, E4M3 pages of a sliding layer.
        _case("append 8 prompts e4m3", "append", layer="sliding", kv="e4m3", q_heads=16, page=32, batch=8, ctx_lo=0,
              ctx_hi=4096, tok_lo=257, tok_hi=2047, fused=True),
        # One sequence at 4096: the latency of one decode layer.
        _case("decode b1 c4096", "attend", ctx_lo=4096, ctx_hi=4096),
        # The batch-64 step's full layer: bandwidth of the page reads.
        _case("decode b64", "attend", batch=64, ctx_lo=512, ctx_hi=32768, sink=True),
        # Group 8, batch 256, E4M3 pages, sinks and output gates.
        _case("decode b256 g8 e4m3", "attend", kv="e4m3", q_heads=16, page=128, batch=256, ctx_lo=512, ctx_hi=8192, sink=True,
              gate=True),
        # A sliding layer of the batch-64 step in small pages: 512 keys of each sequence.
        _case("decode sliding b64", "attend", layer="sliding", page=16, batch=64, ctx_lo=512, ctx_hi=32768, sink=True),
        # Verification of 2 to 7 drafted tokens of 16 sequences.
        _case("tokens b16", "attend", page=32, batch=16, ctx_lo=700, ctx_hi=8192, tok_lo=2, tok_hi=7, gate=True),
        # The last 4096 tokens of a 32768-token prompt.
        _case("chunk 4096 of 32768", "attend", page=64, ctx_lo=28672, ctx_hi=28672, tok_lo=4096, tok_hi=4096, sink=True),
        # Ragged prompts of a sliding layer in pages that end inside every tile.
        _case("prompts sliding", "attend", layer="sliding", page=16, batch=5, ctx_lo=0, ctx_hi=2000, tok_lo=511, tok_hi=4099,
              sink=True),
        # A whole prompt at group 8 over E4M3 pages.
        _case("prompt 8192 g8 e4m3", "attend", kv="e4m3", q_heads=16, page=128, tok_lo=8192, tok_hi=8192),
        # Long contexts: 64 of 2049 pages for each kv head.
        _case("select b4 c131072", "select", batch=4, ctx_lo=131072, ctx_hi=131072, sink=True, pages=64),
        # The batch-64 contexts at group 8 over E4M3 pages: 33 of up to 1025 pages.
        _case("select b64 g8 e4m3", "select", kv="e4m3", q_heads=16, page=32, batch=64, ctx_lo=512, ctx_hi=32768, pages=33),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "select"])
    group = rng.choice([1, 2, 4, 4, 8])
    kv_heads = rng.choice([1, 2, 2, 4])
    c = _case("", op, kv=rng.choice(["bf16", "bf16", "e4m3"]), kv_heads=kv_heads, q_heads=group * kv_heads,
              page=rng.choice([16, 32, 64, 128, 256]), layer=rng.choice(["full", "full", "sliding"]),
              sink=rng.random() < 0.5, gate=op == "attend" and rng.random() < 0.3, fused=op == "append" and rng.random() < 0.5)
    del c["name"]
    c["batch"] = _log(rng, 1, 256)
    if op == "select":
        c["layer"] = "full"
        c["pages"] = _log(rng, 2, 128)
        c["batch"] = _log(rng, 1, 64)
        c["ctx_hi"] = _log(rng, 64, min(131072, (1 << 20) // (c["batch"] * kv_heads)))
        c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
        return c
    kind = rng.choice(["one", "few", "chunk"])
    if kind == "one":
        c["ctx_hi"] = _log(rng, 1, min(131072, (1 << 21) // (c["batch"] * kv_heads)))
    elif kind == "few":
        c["batch"] = _log(rng, 1, 64)
        c["tok_hi"] = rng.randint(2, 9)
        c["tok_lo"] = rng.randint(1, c["tok_hi"])
        c["ctx_hi"] = _log(rng, 1, min(32768, (1 << 19) // (c["batch"] * kv_heads)))
    else:
        c["batch"] = _log(rng, 1, 8)
        heads = c["batch"] * c["q_heads"]   # at most 2^30 scores in all, as the largest listed case has
        c["tok_hi"] = _log(rng, 16, min(8192 // c["batch"], math.isqrt((1 << 29) // heads)))
        c["tok_lo"] = rng.randint(1, c["tok_hi"])
        c["ctx_hi"] = _log(rng, 1, min(32768, (1 << 30) // (heads * c["tok_hi"]) - c["tok_hi"]))
    c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
    return c


def _lengths(c):
    """(previous tokens, new tokens) of every sequence of a case."""
    rng = random.Random(1000 * c["batch"] + c["ctx_hi"] + 7 * c["tok_hi"])
    return ([rng.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["batch"])],
            [rng.randint(c["tok_lo"], c["tok_hi"]) for _ in range(c["batch"])])


def _first_key(c, p):
    return max(0, p - WINDOW + 1) if c["layer"] == "sliding" else 0


def _selected_blocks(c, p):
    """Blocks that a token at position p attends to in a select case."""
    return min(c["pages"], p // c["page"] + 1)


def work(c):
    ctx, tok = _lengths(c)
    e = 1 if c["kv"] == "e4m3" else 2
    rows, Hq, Hkv, ps = sum(tok), c["q_heads"], c["kv_heads"], c["page"]
    tables = 4 * (2 * c["batch"] + 1 + sum(-(-(x + n) // ps) - x // ps for x, n in zip(ctx, tok)))
    if c["op"] == "append":
        rot = ROPE[c["layer"]][0]
        heads = Hq + Hkv
        touched = sum(-(-(x + n) // ps) - x // ps for x, n in zip(ctx, tok))
        reused = sum(x % ps != 0 for x in ctx)   # pages whose bounds are read before they are written
        nbytes = rows * D * (2 * Hq + 4 * Hkv + 2 * Hq + 2 * e * Hkv) + (touched + reused) * Hkv * 2 * D * 2 + tables
        return {"bytes": nbytes + rows * rot * 4, "flops": rows * heads * rot * 3}
    if c["op"] == "attend":
        keys = sum(x + n - _first_key(c, x) for x, n in zip(ctx, tok))   # each read once
        pairs = sum(x + t + 1 - _first_key(c, x + t) for x, n in zip(ctx, tok) for t in range(n))
        nbytes = keys * Hkv * D * 2 * e + rows * Hq * (4 * D + 4 + (4 if c["gate"] else 0))
        return {"bytes": nbytes + 4 * sum(-(-(x + n) // ps) for x, n in zip(ctx, tok)), "flops": pairs * Hq * D * 4}
    blocks = sum(p // ps + 1 for p in ctx)
    chosen = sum(_selected_blocks(c, p) for p in ctx)
    nbytes = blocks * Hkv * 2 * D * 2 + chosen * ps * Hkv * D * 2 * e + rows * Hq * (4 * D + 4) + 4 * (chosen * Hkv + blocks)
    return {"bytes": nbytes, "flops": blocks * Hkv * 4 * D + chosen * ps * Hq * D * 4}


# ------------------------------------------------------------------ inputs --

def _codes(x, scale):
    """E4M3 codes of x / scale (scale per kv head, dim 1), saturating."""
    return (x / scale.view(1, -1, 1, 1).to(x.dtype)).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)


def prepare(case, seed):
    c = dict(_case("", case["op"]), **case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    Hq, Hkv, ps, B = c["q_heads"], c["kv_heads"], c["page"], c["batch"]
    ctx, tok = _lengths(c)
    rows, nblk = sum(tok), -(-max(x + n for x, n in zip(ctx, tok)) // ps)
    off = [0]
    for n in tok:
        off.append(off[-1] + n)
    randn = lambda *shape: torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)  # noqa: E731

    # Which blocks of each sequence hold a page: an append touches only the blocks of its new
    # tokens, a sliding layer only its window; the others' entries name a page that no call reads.
    lo = [x // ps if c["op"] == "append" else _first_key(c, x) // ps for x in ctx]
    hi = [-(-(x + n) // ps) for x, n in zip(ctx, tok)]
    pool = sum(h - w for w, h in zip(lo, hi)) + 3
    order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    blk = torch.arange(nblk, device=dev).unsqueeze(0)
    lo_t, hi_t = torch.tensor(lo, device=dev).unsqueeze(1), torch.tensor(hi, device=dev).unsqueeze(1)
    start = torch.tensor([0] + [h - w for w, h in zip(lo, hi)], device=dev).cumsum(0)[:-1].unsqueeze(1)
    at = torch.where((blk >= lo_t) & (blk < hi_t), start + blk - lo_t, torch.full_like(blk, pool - 1))
    table = order[at].contiguous()

    s = {"case": c, "table": table, "nblk": nblk, "rows": rows, "max_tokens": max(tok), "max_context": max(ctx),
         "context": torch.tensor(ctx, dtype=torch.int32, device=dev), "offsets": torch.tensor(off, dtype=torch.int32, device=dev)}
    seq = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(tok, device=dev))
    s["seq"] = seq                                                  # sequence of each row
    s["tok"] = torch.arange(rows, device=dev) - s["offsets"][seq].long()   # its number among the new tokens
    if c["kv"] == "e4m3":
        s["k_scale"], s["v_scale"] = ((3 + 3 * torch.rand(Hkv, generator=g, device=dev)) / 448 for _ in range(2))
        s["k"] = _codes(randn(pool, Hkv, ps, D), s["k_scale"])
        s["v"] = _codes(randn(pool, Hkv, ps, D), s["v_scale"])
    else:
        s["k_scale"] = s["v_scale"] = None
        s["k"], s["v"] = randn(pool, Hkv, ps, D), randn(pool, Hkv, ps, D)
    if c["op"] == "append":
        if c["fused"]:
            q, k, v = randn(rows, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], dim=1)
        else:
            q, k, v = randn(rows, Hq, D), randn(rows, Hkv, D), randn(rows, Hkv, D)
        s["new"] = (q, k, v)
        s["q_rot"] = torch.empty(rows, Hq, D, dtype=torch.bfloat16, device=dev)
    else:
        s["q"] = randn(rows, Hq, D)
        s["sink"] = torch.randn(Hq, generator=g, device=dev) if c["sink"] else None
        s["gate"] = torch.randn(rows, Hq, generator=g, device=dev) if c["gate"] else None
        s["out"] = torch.empty(rows, Hq, D, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty(rows, Hq, dtype=torch.float32, device=dev)
    if c["op"] == "select":
        # Keys that share a direction within a page, as neighbouring tokens do, so that pages differ.
        if c["kv"] == "bf16":
            s["k"] = s["k"] * 0.7 + randn(pool, Hkv, 1, D)
        s["selected"] = torch.empty(rows, Hkv, c["pages"], dtype=torch.int32, device=dev)
    if c["op"] != "attend":
        # Bounds of the keys that the pages hold so far (an append into a fresh page starts anew).
        used = torch.zeros(pool, dtype=torch.int64, device=dev)
        held = (torch.tensor(ctx, device=dev).unsqueeze(1) + (0 if c["op"] == "append" else 1) - blk * ps).clamp(0, ps)
        used[table.long()[(blk >= lo_t) & (blk < hi_t)]] = held[(blk >= lo_t) & (blk < hi_t)]
        dead = (torch.arange(ps, device=dev) >= used.unsqueeze(1)).view(pool, 1, ps, 1)
        k = s["k"].to(torch.bfloat16)
        s["bounds"] = torch.stack([k.masked_fill(dead, math.inf).amin(2), k.masked_fill(dead, -math.inf).amax(2)], 2).contiguous()
    return s


# ------------------------------------------------------------- plain forms --

def _e4m3_value(x):
    """x (64 bits) rounded once to the nearest E4M3 value, ties to even, saturating."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _rotate(x, pos, layer):
    """Partial rotation of x [rows, heads, 256] by its row's position; the table's cosines and sines have 32 bits."""
    rot, theta = ROPE[layer]
    i = torch.arange(rot // 2, device=x.device, dtype=torch.float64)
    a = pos.double().unsqueeze(1) * theta ** (-2 * i / rot)
    cos, sin = (f(a).float().double().unsqueeze(1) for f in (torch.cos, torch.sin))
    x = x.double()
    x1, x2 = x[..., : rot // 2], x[..., rot // 2: rot]
    return torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin, x[..., rot:]], dim=-1)


def _append(s):
    c = s["case"]
    ps = c["page"]
    q, k, v = s["new"]
    pos = s["context"].long()[s["seq"]] + s["tok"]
    page, slot = s["table"].long()[s["seq"], pos // ps], pos % ps
    s["q_rot"].copy_(_rotate(q, pos, c["layer"]).float())
    k, v = _rotate(k, pos, c["layer"]), v.double()
    if c["kv"] == "e4m3":
        k, v = (_e4m3_value(x / sc.double().view(1, -1, 1)).float().to(torch.float8_e4m3fn)
                for x, sc in ((k, s["k_scale"]), (v, s["v_scale"])))
    else:
        k, v = k.float().to(torch.bfloat16), v.to(torch.bfloat16)
    for_page = lambda t: t.view(torch.uint8) if c["kv"] == "e4m3" else t  # noqa: E731
    for_page(s["k"])[page, :, slot] = for_page(k)
    for_page(s["v"])[page, :, slot] = for_page(v)
    # Bounds: a page whose first slot is written now starts anew; the others keep what they held.
    fresh = torch.zeros(s["k"].shape[0], device=q.device).index_reduce_(0, page, (slot == 0).float(), "amax").view(-1, 1, 1) > 0
    k = k.float()
    lo = torch.where(fresh, math.inf, s["bounds"][:, :, 0].float()).index_reduce_(0, page, k, "amin")
    hi = torch.where(fresh, -math.inf, s["bounds"][:, :, 1].float()).index_reduce_(0, page, k, "amax")
    s["bounds"].copy_(torch.stack([lo, hi], dim=2))
    return {"q": s["q_rot"], "k": s["k"], "v": s["v"], "bounds": s["bounds"]}


def _softmax(score, v, group):
    """Outputs and log-sums of scores [.., kv head, rows, keys] (masked ones at -inf) with values [.., kv head, keys, 256];
    rows are (token, head of the group)."""
    m = score.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(score - m)
    total = p.sum(-1)
    out = (p @ v) / total.unsqueeze(-1)
    lse = m.squeeze(-1) + torch.log(total)
    # [.., kv head, token * group, ..] -> [.., token, q head, ..]
    shape = lse.shape[:-1] + (-1, group)
    lse = lse.reshape(shape).transpose(-3, -2).flatten(-2)
    out = out.reshape(shape + (D,)).transpose(-4, -3).flatten(-3, -2)
    return out, lse


def _finish(out, lse, sink, gate):
    """Rows [rows, q heads, 256] with the sink's share taken off and the output gate applied."""
    if sink is not None:
        out = out * torch.sigmoid(lse - sink).unsqueeze(-1)
    if gate is not None:
        out = out * torch.sigmoid(gate).unsqueeze(-1)
    return out


def _values(t, scale, pages):
    """Slots [batch, kv head, n, slot, 256] of the pages [batch, kv head, n], in 32 bits."""
    head = torch.arange(t.shape[1], device=t.device).view(1, -1, 1)
    x = t.view(torch.uint8)[pages, head].view(t.dtype) if t.dtype == torch.float8_e4m3fn else t[pages, head]
    x = x.float()
    return x if scale is None else x * scale.view(1, -1, 1, 1, 1)


def _attend(s):
    c = s["case"]
    B, N, Hkv, ps, nblk = c["batch"], s["max_tokens"], c["kv_heads"], c["page"], s["nblk"]
    G = c["q_heads"] // Hkv
    dev = s["q"].device
    # The blocks that a sequence's tokens see: all, or those from the first token's window on.
    first, n = torch.zeros(B, 1, device=dev, dtype=torch.long), nblk
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
    start = pos - WINDOW + 1 if c["layer"] == "sliding" else torch.zeros_like(pos)
    seen = (key.unsqueeze(1) <= pos.unsqueeze(-1)) & (key.unsqueeze(1) >= start.unsqueeze(-1))   # [B, N, keys]
    score = (q @ k.transpose(-1, -2)).mul_(1 / 16).view(B, Hkv, N, G, -1)
    score.masked_fill_(~seen.view(B, 1, N, 1, -1), -math.inf)
    out, lse = _softmax(score.view(B, Hkv, N * G, -1), v, G)         # [B, N, Hq, ..]
    out, lse = out[s["seq"], s["tok"]], lse[s["seq"], s["tok"]]
    return {"out": _finish(out, lse, s["sink"], s["gate"]).to(torch.bfloat16), "lse": lse}


def _select(s):
    c = s["case"]
    B, Hkv, ps, nblk, S = c["batch"], c["kv_heads"], c["page"], s["nblk"], c["pages"]
    G = c["q_heads"] // Hkv
    dev = s["q"].device
    # Score of a block: the sum over the group's heads of sum_d max(q_d lo_d, q_d hi_d); in 64 bits, as a
    # choice between near equals has to come out the same.
    q = s["q"].view(B, Hkv, G, D).double()
    b = s["bounds"][s["table"].long()].double()                                            # [B, nblk, Hkv, 2, D]
    score = torch.einsum("bhd,bnhd->bhn", q.clamp(max=0).sum(2), b[:, :, :, 0]) + torch.einsum("bhd,bnhd->bhn", q.clamp(min=0).sum(2), b[:, :, :, 1])
    pos = s["context"].long()
    last = (pos // ps).view(B, 1, 1)
    blk = torch.arange(nblk, device=dev)
    score = torch.where((blk == 0) | (blk == last), math.inf, score)                       # always chosen
    score = torch.where(blk > last, -math.inf, score)
    k = min(S, nblk)
    chosen = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :k]
    chosen = torch.where(chosen > last, nblk, chosen).sort(-1).values                      # ascending, past the end last
    there = chosen < nblk
    selected = torch.full((B, Hkv, S), -1, device=dev, dtype=torch.int32)
    selected[..., :k] = torch.where(there, chosen, -1)
    pages = s["table"].long().unsqueeze(1).expand(B, Hkv, nblk).gather(-1, chosen.clamp(max=nblk - 1))
    kk, vv = (_values(s[n], s[n + "_scale"], pages).flatten(2, 3) for n in ("k", "v"))
    key = (chosen.unsqueeze(-1) * ps + torch.arange(ps, device=dev)).flatten(-2)           # [B, Hkv, keys]
    seen = (key <= pos.view(B, 1, 1)) & there.unsqueeze(-1).expand(B, Hkv, k, ps).flatten(-2)
    x = (s["q"].float().view(B, Hkv, G, D) @ kk.transpose(-1, -2)) / 16
    out, lse = _softmax(x.masked_fill(~seen.unsqueeze(2), -math.inf), vv, G)
    out, lse = out[:, 0], lse[:, 0]
    return {"selected": selected, "out": _finish(out, lse, s["sink"], None).to(torch.bfloat16), "lse": lse}


# ------------------------------------------------------ the framework's way --

@functools.lru_cache(maxsize=None)
def _context(q_heads, kv_heads, kv):
    """The context that a serving program keeps for its model: one sliding and one full layer here."""
    import full_gqa_decode_gb300 as hd
    return hd.hybrid_decode_init(hd.Config(layer_types=[hd.HD_SLIDING, hd.HD_FULL], num_q_heads=q_heads, num_kv_heads=kv_heads,
                                           sliding_window=WINDOW, max_batch=MAX_BATCH, max_context=MAX_CONTEXT,
                                           kv_dtype=hd.HD_KV_FP8_E4M3 if kv == "e4m3" else hd.HD_KV_BF16))


def _plan(s):
    """Descriptors of the batch and the cache, made once for a step's tensors."""
    import full_gqa_decode_gb300 as hd
    c = s["case"]
    offsets = None if c["tok_hi"] == 1 else s["offsets"]
    return (hd, _context(c["q_heads"], c["kv_heads"], c["kv"]), int(c["layer"] == "full"),
            hd.paged_batch(s["table"], s["context"], offsets, num_tokens=s["rows"], max_tokens=s["max_tokens"],
                           max_context=s["max_context"]),
            hd.paged_cache(s["k"], s["v"], s["k_scale"], s["v_scale"], bounds=s.get("bounds")))


def _own(s):
    if "plan" not in s:
        s["plan"] = _plan(s)
    hd, ctx, layer, batch, cache = s["plan"]
    op = s["case"]["op"]
    if op == "append":
        hd.rope_append_paged(ctx, layer, batch, *s["new"], s["q_rot"], cache)
        return {"q": s["q_rot"], "k": s["k"], "v": s["v"], "bounds": s["bounds"]}
    if op == "attend":
        hd.attn_paged(ctx, layer, batch, s["q"], cache, s["sink"], s["out"], s["lse"], gate=s["gate"])
        return {"out": s["out"], "lse": s["lse"]}
    hd.select_pages(ctx, layer, batch, s["q"], cache, s["selected"], keep_first=1, keep_last=1)
    hd.attn_selected_pages(ctx, layer, batch, s["q"], cache, s["selected"], s["sink"], s["out"], s["lse"])
    return {"selected": s["selected"], "out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"append": _append, "attend": _attend, "select": _select}[state["case"]["op"]](state)


# ------------------------------------------------------- 64-bit definitions --

def _exact_rows(q, keys, values, allowed, scale_k, scale_v):
    """softmax(q k / 16) v in 64 bits for q [heads, 256] of one token or [tokens, heads, 256] over keys [n, 256];
    allowed [tokens, n]."""
    s = torch.einsum("thd,nd->thn", q.double(), keys.double()) * (scale_k / 16)
    s = s.masked_fill(~allowed.unsqueeze(1), -math.inf)
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - lse.unsqueeze(-1))
    return torch.einsum("thn,nd->thd", w, values.double()) * scale_v, lse


def _exact_append(s):
    c = s["case"]
    ps, (rot, theta) = c["page"], ROPE[c["layer"]]
    q, k, v = (x.double().clone() for x in s["new"])
    pos = torch.cat([torch.arange(x, x + n, device=q.device) for x, n in zip(*_lengths(c))])
    freq = torch.exp(torch.arange(0, rot, 2, device=q.device, dtype=torch.float64) * (-math.log(theta) / rot))
    turn = torch.polar(torch.ones((), device=q.device, dtype=torch.float64), pos.double().unsqueeze(1) * freq).unsqueeze(1)
    for x in (q, k):
        z = torch.complex(x[..., : rot // 2].contiguous(), x[..., rot // 2: rot].contiguous()) * turn
        x[..., : rot // 2], x[..., rot // 2: rot] = z.real, z.imag
    if c["kv"] == "e4m3":   # codes go by one rounding of 32-bit cosines: the plain form's to say
        return {"q": q, "k": None, "v": None, "bounds": None}
    pages = [s["k"].double(), s["v"].double()]
    r = 0
    for b, (x, n) in enumerate(zip(*_lengths(c))):
        for t in range(n):
            page = int(s["table"][b, (x + t) // ps])
            pages[0][page, :, (x + t) % ps] = k[r]
            pages[1][page, :, (x + t) % ps] = v[r]
            r += 1
    return {"q": q, "k": pages[0], "v": pages[1], "bounds": None}


def _exact_attend(s):
    c = s["case"]
    ps, Hkv = c["page"], c["kv_heads"]
    G = c["q_heads"] // Hkv
    out = torch.empty(s["rows"], c["q_heads"], D, dtype=torch.float64, device=s["q"].device)
    lse = torch.empty(s["rows"], c["q_heads"], dtype=torch.float64, device=s["q"].device)
    r0 = 0
    for b, (x, n) in enumerate(zip(*_lengths(c))):
        w0 = _first_key(c, x) // ps * ps
        pages = s["table"][b, w0 // ps: -(-(x + n) // ps)].long()
        for h in range(Hkv):
            key, val = ((t.view(torch.uint8)[pages, h].view(t.dtype) if c["kv"] == "e4m3" else t[pages, h]).flatten(0, 1)[: x + n - w0] for t in (s["k"], s["v"]))
            sk, sv = (1.0, 1.0) if s["k_scale"] is None else (float(s["k_scale"][h]), float(s["v_scale"][h]))
            for t0 in range(0, n, 512):
                p = torch.arange(x + t0, x + min(n, t0 + 512), device=key.device).unsqueeze(1)
                at = torch.arange(w0, x + n, device=key.device)
                ok = (at <= p) & ((at > p - WINDOW) | (c["layer"] == "full"))
                rows = slice(r0 + t0, r0 + min(n, t0 + 512))
                hs = slice(h * G, h * G + G)
                out[rows, hs], lse[rows, hs] = _exact_rows(s["q"][rows, hs], key, val, ok, sk, sv)
        r0 += n
    if s["sink"] is not None:
        out /= 1 + torch.exp(s["sink"].double() - lse).unsqueeze(-1)
    if s["gate"] is not None:
        out /= 1 + torch.exp(-s["gate"].double()).unsqueeze(-1)
    return {"out": out, "lse": lse}


def _exact_select(s):
    c = s["case"]
    ps, Hkv, S = c["page"], c["kv_heads"], c["pages"]
    G = c["q_heads"] // Hkv
    q = s["q"]
    selected = torch.full((c["batch"], Hkv, S), -1, dtype=torch.int64, device=q.device)
    out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
    for b, p in enumerate(_lengths(c)[0]):
        n = p // ps + 1
        pages = s["table"][b, :n].long()
        for h in range(Hkv):
            hs = slice(h * G, h * G + G)
            bound = torch.maximum(q[b, hs].double().unsqueeze(1) * s["bounds"][pages, h, 0].double(),
                                  q[b, hs].double().unsqueeze(1) * s["bounds"][pages, h, 1].double()).sum((0, 2))
            bound[0] = bound[n - 1] = math.inf
            pick = torch.argsort(-bound, stable=True)[:S].sort().values
            selected[b, h, : len(pick)] = pick
            at = (pick.unsqueeze(1) * ps + torch.arange(ps, device=q.device)).flatten()
            key, val = ((t.view(torch.uint8)[pages[pick], h].view(t.dtype) if c["kv"] == "e4m3" else t[pages[pick], h]).flatten(0, 1)[at <= p] for t in (s["k"], s["v"]))
            sk, sv = (1.0, 1.0) if s["k_scale"] is None else (float(s["k_scale"][h]), float(s["v_scale"][h]))
            o, ls = _exact_rows(q[b: b + 1, hs], key, val, torch.ones(1, len(key), dtype=torch.bool, device=q.device), sk, sv)
            out[b, hs], lse[b, hs] = o[0], ls[0]
    if s["sink"] is not None:
        out /= 1 + torch.exp(s["sink"].double() - lse).unsqueeze(-1)
    return {"selected": selected, "out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "select": _exact_select}[s["case"]["op"]](s)
