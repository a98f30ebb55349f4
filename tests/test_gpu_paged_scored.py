"""GPU tests of attn_paged_scored against 64-bit references: caps, biases,
documents, prefixes and blocks, alone and together, for single tokens, few and
chunks; rows that see nothing, lists that do not ascend, extremes, capture,
streams, and a step of normed append, attention and reading back."""
import numpy as np
import pytest
import torch

import synth
from paged_harness import D, PagedCase, assert_rows, reference_rows
from scored_harness import Rule, documents, prefixes, reference_scored, slopes_of, visible
from test_gpu_paged import cache_of, context, sinks

pytestmark = pytest.mark.gpu
INT_MIN, INT_MAX = -2 ** 31, 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def run(hd, ctx, case, rule, d=None, sink=None, gate=None, **kw):
    d = d or case.device()
    out = torch.full((case.rows, case.q_heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((case.rows, case.q_heads), 7.0, device="cuda")
    sink_d, gate_d = (None if t is None else t.cuda() for t in (sink, gate))
    hd.attn_paged_scored(ctx, 0 if case.window else 1, case.batch_of(hd, d, **kw), rule.device(hd), d["q"], cache_of(hd, d), sink_d,
                         out, lse, gate=gate_d)
    torch.cuda.synchronize()
    return out, lse


def check(hd, orc, case, rule, rows=None, sink=None, gate=None, ctx=None, errors=0, **kw):
    ctx = ctx or context(hd, case.group, case.kv_heads, case.kv, window=case.window or 512)
    out, lse = run(hd, ctx, case, rule, sink=sink, gate=gate, **kw)
    assert hd.hybrid_decode_device_errors(ctx) == errors
    assert_rows(reference_scored(orc, case, rule, rows, sink, gate), out, lse)
    return out, lse


SPANS = {
    "single": [(0, 1), (1, 1), (15, 1), (16, 1), (63, 1), (64, 1), (700, 1), (2047, 1), (5, 1)],
    "few": [(0, 2), (5, 0), (63, 2), (250, 2), (511, 1), (1000, 2)],
    "chunks": [(0, 150), (63, 5), (300, 90), (7, 0), (700, 33)],
}
RULES = ("cap", "distance", "documents", "prefix", "blocks", "all")


def rule_of(name, case):
    if name == "cap":
        return Rule(softcap=30.0)
    if name == "distance":
        return Rule(slopes=slopes_of(case.q_heads))
    if name == "documents":
        return Rule(first=documents(case, [20, 3, 1, 64]))
    if name == "prefix":
        return Rule(last=prefixes(case, [40, 0, 320, 1, 2000]))
    # Blocks that see themselves whole and nothing else; with everything else.
    first = documents(case, [13, 50, 2])
    last = np.concatenate([np.array([x + np.searchsorted(first[a:b], first[a:b][i], side="right") - 1 for i in range(b - a)], np.int64)
                           for (x, _), a, b in zip(case.spans, case.offsets, case.offsets[1:])])
    if name == "blocks":
        return Rule(first=first, last=last)
    return Rule(softcap=20.0, scale=0.25, slopes=slopes_of(case.q_heads, 0.3), first=first, last=last)


@pytest.mark.parametrize("name", RULES)
@pytest.mark.parametrize("spans", sorted(SPANS))
@pytest.mark.parametrize("group,kv,page,window", [(4, "bf16", 64, 0), (8, "e4m3", 32, 0), (1, "bf16", 16, 100), (2, "e4m3", 128, 512)])
def test_rules(hd, orc, name, spans, group, kv, page, window):
    case = PagedCase(201, SPANS[spans], group=group, kv=kv, page=page, window=window, single=spans == "single")
    case.q *= 4
    check(hd, orc, case, rule_of(name, case), sink=sinks(case) if group == 4 else None,
          gate=synth.normal_bf16(case.rng, (case.rows, case.q_heads)).float() if group == 8 else None)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows", [128, 132])   # at group 4: all of one CTA's rows, and a few of its peer
def test_tiles_of_one_cta_and_just_more(hd, orc, kv, rows):
    case = PagedCase(202, [(90, rows // 4), (0, rows // 4)], kv=kv)
    check(hd, orc, case, rule_of("all", case))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_prefix_longer_than_a_tile_of_queries(hd, orc, kv):
    """Queries of the first tiles see keys of later ones; the prefix ends inside a tile and past the sequence."""
    case = PagedCase(203, [(0, 300), (50, 250), (0, 130)], kv=kv, page=16)
    check(hd, orc, case, Rule(last=prefixes(case, [217, 290, 4000])), rows=range(0, case.rows, 7))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_documents_of_a_long_prompt(hd, orc, kv):
    """Tiles that start far inside the sequence, and whole tiles in one document."""
    case = PagedCase(204, [(3000, 1500)], kv=kv, page=64)
    check(hd, orc, case, Rule(first=documents(case, [700, 5, 130, 64, 256])), rows=range(0, case.rows, 13))


@pytest.mark.parametrize("n", [1, 2, 70])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_rows_that_see_nothing(hd, orc, kv, n):
    """Out 0 and lse -inf, with sinks and gates, beside rows that see something; whole tiles of such rows among them."""
    case = PagedCase(205, [(0, n), (300, n), (40, n), (511, n)], kv=kv, single=n == 1)
    first = np.concatenate([np.arange(c, c + n) for c, _ in case.spans]) - 3
    first[: n] = 10 ** 6                       # all of the first sequence
    first[2 * n: 3 * n] = np.where(np.arange(n) < n // 2, 0, INT_MAX)
    gate = synth.normal_bf16(case.rng, (case.rows, case.q_heads)).float()
    rule = Rule(first=first)
    out, lse = check(hd, orc, case, rule, sink=sinks(case), gate=gate)
    for r in range(case.rows):
        _, lo, hi = visible(case, rule, r)
        if hi < lo:
            assert (out[r] == 0).all() and torch.isneginf(lse[r]).all()
    # The same by their ends.
    last = np.concatenate([np.arange(c, c + n) for c, _ in case.spans])
    last[: n] = INT_MIN
    last[n: 2 * n] = -1
    rule = Rule(softcap=30.0, last=last)
    out, lse = check(hd, orc, case, rule, sink=sinks(case), gate=gate)
    assert (out[: 2 * n] == 0).all() and torch.isneginf(lse[: 2 * n]).all()


@pytest.mark.parametrize("n", [1, 70])
def test_pages_that_no_row_sees_are_not_needed(hd, orc, n):
    """Entries of the block table before every row's first position, and behind its last, may be anything."""
    case = PagedCase(206, [(500, n), (900, n)], single=n == 1, page=32)
    first = np.concatenate([np.full(n, 450), np.full(n, 10 ** 6)])
    d = case.device()
    d["table"][0, : 450 // 32] = 2 ** 30
    d["table"][1, :] = -5
    check(hd, orc, case, Rule(first=first), d=d)


def test_lists_that_do_not_ascend_are_flagged(hd, orc):
    """Rows that their tile would not serve right are NaN; the others, and the other sequences, are as they should be."""
    for n in (2, 64):
        case = PagedCase(207, [(300, n), (100, n)])
        first = np.zeros(case.rows, np.int64)
        first[n // 2 - (n == 2)] = 250           # above the last row's
        ctx = context(hd)
        rule = Rule(first=first)
        out, lse = run(hd, ctx, case, rule)
        assert hd.hybrid_decode_device_errors(ctx) == 64
        ref = reference_scored(orc, case, rule)
        bad = [r for r in range(case.rows) if torch.isnan(lse[r]).any()]
        assert bad and all(r < n for r in bad)
        assert torch.isnan(out[bad].float()).all() and torch.isnan(lse[bad]).all()
        assert_rows({r: ref[r] for r in range(case.rows) if r not in bad}, out, lse)


@pytest.mark.parametrize("spans", sorted(SPANS))
@pytest.mark.parametrize("cap", [1.0 / 1024, 1.0, 1024.0])
def test_extreme_caps(hd, orc, spans, cap):
    case = PagedCase(208, SPANS[spans], single=spans == "single")
    case.q *= 40
    check(hd, orc, case, Rule(softcap=cap))


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_scores_far_beyond_the_cap(hd, orc, kv, n):
    """Scores of 10^18 and more: the exponential overflows and underflows, the cap holds."""
    case = PagedCase(209, [(200, n), (31, n)], kv=kv, single=n == 1)
    case.q *= 1e18
    ctx = context(hd, kv=kv)
    out, lse = run(hd, ctx, case, Rule(softcap=50.0))
    assert hd.hybrid_decode_device_errors(ctx) == 0
    # Scores are +-50 to the last bit of a tanh: the sign alone counts.
    for r in (0, case.rows - 1):
        b, p = case.token(r)
        for h in range(case.kv_heads):
            k = case.entries(orc, case.k, case.k_scale, h, case.table[b, : -(-sum(case.spans[b]) // case.page)])[: p + 1]
            v = case.entries(orc, case.v, case.v_scale, h, case.table[b, : -(-sum(case.spans[b]) // case.page)])[: p + 1]
            s = case.q[r, h * 4: h * 4 + 4].double().numpy() @ k.T
            w = (s > 0).astype(float)
            unsure = (np.abs(s) < 2.0 ** -16 * (np.abs(case.q[r, h * 4: h * 4 + 4].double().numpy()) @ np.abs(k).T)).sum(1, keepdims=True)
            assert (w.sum(1) > 0).all() and (unsure <= 1).all()
            unsure = 2.0 * unsure / w.sum(1, keepdims=True)   # a score whose sign the fp32 sum may not tell
            want = (w @ v) / w.sum(1, keepdims=True)
            A = (w @ np.abs(v)) / w.sum(1, keepdims=True)
            got = out[r, h * 4: h * 4 + 4].double().cpu().numpy()
            assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.2 * 2.0 ** -20 * 51) * A + unsure * np.abs(v).max()).all()
            off = np.abs(lse[r, h * 4: h * 4 + 4].double().cpu().numpy() - 50 - np.log(w.sum(1)))
            assert (off < 1.1 * 2.0 ** -20 * 51 + 2.0 ** -15 + unsure[:, 0]).all()


@pytest.mark.parametrize("n", [1, 60])
def test_steep_and_negative_slopes(hd, orc, n):
    """Slopes of either sign and zero: the far keys win, or only the nearest counts."""
    case = PagedCase(210, [(1000, n), (90, n)], single=n == 1, kv_heads=2)
    slopes = np.array([0.0, -0.01, 5.0, 100.0, -1.0, 1e-4, 0.5, -0.25], np.float32)
    check(hd, orc, case, Rule(slopes=slopes), rows=range(0, case.rows, 7))
    check(hd, orc, case, Rule(slopes=slopes, softcap=10.0), rows=range(0, case.rows, 7))


def test_long_context_in_many_pieces(hd, orc):
    """Items cut between CTAs, single tokens and chunks, with everything at once."""
    for spans in ([(19000, 1), (300, 1)], [(9000, 70), (5, 20)]):
        for kv in ("bf16", "e4m3"):
            case = PagedCase(211, spans, kv=kv, single=spans[0][1] == 1)
            case.q *= 3
            rule = Rule(softcap=20.0, slopes=slopes_of(case.q_heads, 0.05), first=np.where(np.arange(case.rows) < spans[0][1], 120, 0))
            check(hd, orc, case, rule, rows=range(0, case.rows, 9), sink=sinks(case))


def test_no_rule_is_attn_paged(hd, orc):
    for spans in ("single", "chunks"):
        case = PagedCase(212, SPANS[spans], single=spans == "single")
        ctx = context(hd)
        out, lse = run(hd, ctx, case, Rule())
        assert_rows(reference_rows(orc, case), out, lse)
        d = case.device()
        a, b = (torch.empty(case.rows, case.q_heads, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        ls = torch.empty(case.rows, case.q_heads, device="cuda")
        import ctypes
        batch, cache = case.batch_of(hd, d), cache_of(hd, d)
        hd.attn_paged(ctx, 1, batch, d["q"], cache, None, a, ls)
        assert hd._lib.attn_paged_scored(ctx.handle, 1, batch.ref, None, d["q"].data_ptr(), cache.ref, None, None, b.data_ptr(),
                                         ls.data_ptr(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
        torch.cuda.synchronize()
        assert torch.equal(a, b), "no rule at all: the same kernel"


def test_rows_of_no_sequence_stay_and_bad_sequences_are_nan(hd, orc):
    case = PagedCase(213, [(0, 4), (5, 3), (90, 9)])
    d = case.device()
    d["context"][1] = -3
    rule = Rule(softcap=30.0, first=np.zeros(case.rows + 2, np.int64))
    q = torch.cat([d["q"], d["q"][:2]])
    out = torch.full((case.rows + 2, case.q_heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((case.rows + 2, case.q_heads), 7.0, device="cuda")
    ctx = context(hd)
    hd.attn_paged_scored(ctx, 1, case.batch_of(hd, d, num_tokens=case.rows + 2), rule.device(hd), q, cache_of(hd, d), None, out, lse)
    torch.cuda.synchronize()
    assert hd.hybrid_decode_device_errors(ctx) == 1
    assert (out[case.rows:] == 7).all() and (lse[case.rows:] == 7).all()
    assert torch.isnan(out[4:7].float()).all() and torch.isnan(lse[4:7]).all()
    assert_rows({r: x for r, x in reference_scored(orc, case, rule).items() if not 4 <= r < 7}, out[: case.rows], lse[: case.rows])


@pytest.mark.parametrize("long_one", [False, True])
def test_more_sequences_than_a_warp(hd, orc, long_one):
    rng = np.random.default_rng(3)
    spans = [(int(c), int(n)) for c, n in zip(rng.integers(0, 300, 60), rng.integers(0, 3, 60))]
    if long_one:
        spans[17] = (40, 400)
    case = PagedCase(214, spans, page=16)
    check(hd, orc, case, rule_of("all", case), rows=range(0, case.rows, 5))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_more_sequences_than_a_block_has_threads(hd, orc, kv):
    """Single tokens of 300 sequences, some of which see nothing, and a chunk among them."""
    rng = np.random.default_rng(4)
    for spans in ([(int(c), 1) for c in rng.integers(0, 150, 300)],
                  [(int(c), int(n)) for c, n in zip(rng.integers(0, 60, 400), rng.integers(0, 2, 400))] + [(30, 260)]):
        single = len(spans) == 300
        case = PagedCase(223, spans, kv=kv, page=16, single=single)
        first = np.concatenate([np.full(n, c + n if i % 7 == 3 else max(0, c - 20)) for i, (c, n) in enumerate(spans)])
        ctx = context(hd, kv=kv, max_batch=512)
        check(hd, orc, case, Rule(softcap=10.0, first=first), rows=range(0, case.rows, 3), ctx=ctx, max_context=200)


@pytest.mark.parametrize("n", [1, 50])
def test_captured_and_replayed_on_another_stream(hd, orc, n):
    """A captured call takes new queries, contexts and lists from the same tensors."""
    case = PagedCase(215, [(400, n), (33, n)], single=n == 1)
    ctx, d = context(hd), case.device()
    stream = torch.cuda.Stream()
    first = torch.zeros(case.rows, dtype=torch.int32, device="cuda")
    rule = hd.scoring(softcap=25.0, first=first)
    out, lse = torch.empty_like(d["q"]), torch.empty(case.rows, case.q_heads, device="cuda")
    q = d["q"].clone()
    batch, cache = case.batch_of(hd, d, max_context=1000), cache_of(hd, d)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        hd.attn_paged_scored(ctx, 1, batch, rule, q, cache, None, out, lse)   # set-up outside the capture
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            hd.attn_paged_scored(ctx, 1, batch, rule, q, cache, None, out, lse)
        for k in range(2):
            lists = np.full(case.rows, 10 * k, np.int64)
            first.copy_(torch.from_numpy(lists.astype(np.int32)))
            q.copy_(d["q"] * (k + 1))
            graph.replay()
            stream.synchronize()
            case_k = PagedCase(215, [(400, n), (33, n)], single=n == 1)
            case_k.q = q.cpu()
            assert_rows(reference_scored(orc, case_k, Rule(softcap=25.0, first=lists)), out, lse)
    assert hd.hybrid_decode_device_errors(ctx) == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,stage", [(1, 5), (70, 3)])
def test_lost_copies_time_out_and_the_context_recovers(hd, orc, kv, n, stage):
    case = PagedCase(216, [(19000, n), (300, n), (9000, n), (18000, n)] * (2 if n == 1 else 1), kv=kv, single=n == 1)
    ctx, d, rule = context(hd, kv=kv), case.device(), rule_of("cap", case)
    rows = range(0, case.rows, 17)
    check(hd, orc, case, rule, rows=rows, d=d)
    hd.hybrid_decode_inject_lost_copy(ctx, stage)
    try:
        run(hd, ctx, case, rule, d=d)
    finally:
        hd.hybrid_decode_inject_lost_copy(ctx, -1)
    assert hd.hybrid_decode_device_errors(ctx) == 8
    check(hd, orc, case, rule, rows=rows, d=d)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [0, 512])
def test_prompt_in_parts_equals_one_prompt(hd, orc, kv, window):
    """A capped prompt of packed documents in three calls and token by token sees what it sees in one."""
    whole = PagedCase(217, [(0, 330)], kv=kv, window=window, page=16)
    rule = Rule(softcap=20.0, slopes=slopes_of(whole.q_heads, 0.1), first=documents(whole, [100, 37, 150]))
    ctx, d = context(hd, kv=kv), whole.device()
    ref = reference_scored(orc, whole, rule)
    at = 0
    for n in (150, 1, 1, 2, 176):
        part = hd.paged_batch(d["table"], torch.tensor([at], dtype=torch.int32, device="cuda"),
                              torch.tensor([0, n], dtype=torch.int32, device="cuda"), num_tokens=n, max_tokens=n)
        out = torch.empty(n, whole.q_heads, D, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(n, whole.q_heads, device="cuda")
        sub = Rule(rule.softcap, 0.0, rule.slopes, rule.first[at: at + n])
        hd.attn_paged_scored(ctx, 0 if window else 1, part, sub.device(hd), d["q"][at: at + n].contiguous(), cache_of(hd, d), None, out, lse)
        torch.cuda.synchronize()
        assert_rows({r - at: x for r, x in ref.items() if at <= r < at + n}, out, lse)
        at += n
    assert at == 330 and hd.hybrid_decode_device_errors(ctx) == 0


@pytest.mark.parametrize("n", [1, 12, 90])   # the decode kernel's one tile, several, and the chunk kernel
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_offsets_past_32_bits(hd, orc, kv, n):
    """Pages whose offsets in elements pass 2^31."""
    case = PagedCase(219, [(300, n), (40, n)], kv=kv, page=256, kv_heads=1, group=4, single=n == 1)
    big = 2 ** 31 // (256 * 256) + 40
    k, v = (torch.zeros(big, 1, 256, D, dtype=t.dtype, device="cuda") for t in (case.k, case.v))
    k[big - case.pool:], v[big - case.pool:] = case.k.cuda(), case.v.cuda()
    d = case.device()
    ctx = context(hd, 4, 1, kv)
    cache = hd.paged_cache(k, v, d["k_scale"], d["v_scale"])
    batch = hd.paged_batch((d["table"] + (big - case.pool)).contiguous(), d["context"], d["offsets"], num_tokens=case.rows,
                           max_tokens=case.max_tokens, max_context=300)
    out, lse = torch.empty_like(d["q"]), torch.empty(case.rows, case.q_heads, device="cuda")
    rule = rule_of("all", case)
    hd.attn_paged_scored(ctx, 1, batch, rule.device(hd), d["q"], cache, None, out, lse)
    torch.cuda.synchronize()
    assert hd.hybrid_decode_device_errors(ctx) == 0
    assert_rows(reference_scored(orc, case, rule, rows=range(0, case.rows, 5)), out, lse)


@pytest.mark.parametrize("n", [1, 60])
def test_two_contexts_at_once(hd, orc, n):
    """Calls of two contexts on two streams, each with its own workspace."""
    cases = [PagedCase(220 + i, [(2500 - 300 * i, n), (40, n), (700, n)], single=n == 1) for i in range(2)]
    rules = [Rule(softcap=20.0), Rule(slopes=slopes_of(8), first=documents(cases[1], [50, 9]))]
    ctxs = [hd.hybrid_decode_init(hd.Config(layer_types=[0, 1], max_batch=8, max_context=4000)) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    d = [c.device() for c in cases]
    outs = [(torch.empty_like(x["q"]), torch.empty(c.rows, 8, device="cuda")) for c, x in zip(cases, d)]
    on = [r.device(hd) for r in rules]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            hd.attn_paged_scored(ctxs[i], 1, cases[i].batch_of(hd, d[i]), on[i], d[i]["q"], cache_of(hd, d[i]), None, *outs[i],
                                 stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert hd.hybrid_decode_device_errors(ctxs[i]) == 0
        assert_rows(reference_scored(orc, cases[i], rules[i], rows=range(0, cases[i].rows, 7)), *outs[i])
        ctxs[i].close()


@pytest.mark.parametrize("tokens", [3, 9, 40, 41])   # at group 4: 12 to 164 rows, on both sides of the choice of kernel
@pytest.mark.parametrize("contexts", [(0, 7, 100), (2600, 300, 1900)])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_calls_of_few_rows(hd, orc, kv, contexts, tokens):
    case = PagedCase(222, [(c, tokens - i) for i, c in enumerate(contexts)], kv=kv, page=32)
    check(hd, orc, case, rule_of("all", case), rows=range(0, case.rows, 3), sink=sinks(case), max_context=max(contexts) or 1)


def test_refusals(hd):
    case = PagedCase(218, [(5, 2), (7, 1)])
    ctx, d = context(hd), case.device()
    batch, cache = case.batch_of(hd, d), cache_of(hd, d)
    out, lse = torch.empty_like(d["q"]), torch.empty(case.rows, case.q_heads, device="cuda")

    def call(**kw):
        hd.attn_paged_scored(ctx, 1, batch, hd.scoring(**kw), d["q"], cache, None, out, lse)

    for kw, status in (({"softcap": -1.0}, 1), ({"softcap": float("nan")}, 1), ({"softcap": float("inf")}, 1), ({"scale": -1.0}, 1),
                       ({"scale": float("inf")}, 1), ({"softcap": 1e-4}, 2), ({"softcap": 2000.0}, 2), ({"scale": 1e-10}, 2),
                       ({"scale": 1e10}, 2)):
        with pytest.raises(hd.HDError) as e:
            call(**kw)
        assert e.value.status == status, kw
    ints = torch.zeros(case.rows, dtype=torch.int32, device="cuda")
    for kw in ({"slopes": torch.zeros(case.q_heads + 1, device="cuda")}, {"slopes": torch.zeros(case.q_heads)},
               {"slopes": torch.zeros(case.q_heads, device="cuda").bfloat16()}, {"first": ints[:-1]}, {"last": ints.long()},
               {"last": ints.cpu()}):
        with pytest.raises(ValueError):
            call(**kw)
    call(first=ints, last=ints + 9, slopes=torch.zeros(case.q_heads, device="cuda"), softcap=1024.0, scale=1.0)
    torch.cuda.synchronize()
    assert hd.hybrid_decode_device_errors(ctx) == 0
