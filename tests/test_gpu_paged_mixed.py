"""Calls that a serving program makes of the paged caches: running sequences at
the end of the range next to new prompts, bounds on either side of the choice of
kernel, and paged calls between steps over per-sequence caches."""
import numpy as np
import pytest
import torch

import synth
from harness import FULL, SLIDING, assert_bits_equal
from paged_harness import D, PagedCase, assert_rows, reference_append, reference_rows
from test_gpu_paged import cache_of, context, page_bounds, reference_selection, run_attn, sinks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_running_sequences_at_the_end_of_the_range_beside_a_prompt(hd, orc, kv):
    """Without a max_context of the call's own, every token up to the context's last position is served."""
    case = PagedCase(130, [(1000, 1), (0, 300), (990, 11), (3, 1), (999, 2), (701, 300)], page=16, kv=kv, appended=False)
    ctx, d = context(hd, kv=kv, max_context=1000), case.device()
    k, v = (synth.normal_bf16(case.rng, (case.rows, 2, D)) for _ in range(2))
    held = page_bounds(case)
    held = torch.where(torch.isinf(held), torch.tensor(float("nan"), dtype=torch.bfloat16), held)
    kp, vp, bd, qr = reference_append(orc, case, FULL, case.q, k, v, held)
    bounds, q_rot = held.cuda(), torch.zeros_like(d["q"])
    batch, cache = case.batch_of(hd, d), cache_of(hd, d, bounds)
    hd.rope_append_paged(ctx, 1, batch, d["q"], k.cuda(), v.cuda(), q_rot, cache)
    assert hd.hybrid_decode_device_errors(ctx) == 0
    assert_bits_equal(d["k"], kp, "K pages")
    assert_bits_equal(d["v"], vp, "V pages")
    assert_bits_equal(q_rot, qr, "rotated queries")
    case.k, case.v = d["k"].cpu(), d["v"].cpu()
    rows = [0, 1, 150, 300, 301, 305, 311, 312, 313, 314, 315, 500, 614]
    out, lse = run_attn(hd, ctx, case, d)
    assert_rows(reference_rows(orc, case, rows), out, lse)
    selected = torch.empty(case.rows, 2, 5, dtype=torch.int32, device="cuda")
    hd.select_pages(ctx, 1, batch, d["q"], cache, selected)
    assert np.array_equal(selected.cpu().numpy(), reference_selection(case, torch.from_numpy(bd), 5, 1, 1))
    assert hd.hybrid_decode_device_errors(ctx) == 0
    # one position further is past the tables
    case.spans[2] = (991, 11)
    d["context"][2] = 991
    run_attn(hd, ctx, case, d)
    assert hd.hybrid_decode_device_errors(ctx) == 4


@pytest.mark.parametrize("max_tokens", [4, 40])   # single kernel of few rows, and the one of chunks
def test_rows_that_bad_offsets_name_are_nan(hd, orc, max_tokens):
    """Offsets that leave the tensors: the sequence's rows inside them, and no others."""
    case = PagedCase(131, [(100, 3), (50, 2), (200, 4)], group=1 if max_tokens == 4 else 4)
    ctx, d = context(hd, case.group), case.device()
    bounds = page_bounds(case)
    want = reference_selection(case, bounds, 3, 1, 1)
    for offs, bad in (([0, 3, 5, 900], range(5, 9)), ([-4, 3, 5, 9], range(0, 3)), ([0, 3, 5, -1], range(0))):
        d["offsets"] = torch.tensor(offs, dtype=torch.int32, device="cuda")
        out, lse = run_attn(hd, ctx, case, d, max_tokens=max_tokens)
        assert hd.hybrid_decode_device_errors(ctx) == 16, offs
        selected = torch.full((case.rows, 2, 3), 99, dtype=torch.int32, device="cuda")
        hd.select_pages(ctx, 1, case.batch_of(hd, d, max_tokens=max_tokens), d["q"], cache_of(hd, d, bounds.cuda()), selected)
        assert hd.hybrid_decode_device_errors(ctx) == 16, offs
        for r in range(case.rows):
            if r in bad:
                assert torch.isnan(out[r].float()).all() and torch.isnan(lse[r]).all() and (selected[r] == -1).all()
        good = [r for r in range(5 if offs[3] != 9 else 9) if r not in bad]
        assert_rows(reference_rows(orc, case, good), out, lse)
        assert np.array_equal(selected[good].cpu().numpy(), want[good])


def test_a_context_takes_no_memory_of_its_own_for_paged_calls(hd):
    """The paged calls' workspace is the split-K partials': rows of 1032 bytes, 32 per kv head for each of a full batch's
    2048-key chunks and four more per SM."""
    kw = dict(layer_types=[FULL], num_q_heads=8, num_kv_heads=2, max_batch=16, max_context=4096)
    hd.hybrid_decode_init(hd.Config(**kw)).close()
    before = torch.cuda.mem_get_info()[0]
    ctx = hd.hybrid_decode_init(hd.Config(**kw))
    taken = before - torch.cuda.mem_get_info()[0]
    ctx.close()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    partials = (16 * 3 + 4 * sms) * 2 * 32 * 1032
    tables = 4097 * 32 * 8
    assert taken <= partials + tables + (8 << 20), (taken, partials, tables)   # and little else, in pieces of 2 MB


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("fused", [True, False])
def test_steps_and_paged_calls_take_turns_on_a_stream(hd, kv, fused):
    """decode_step (one grid, or layers as programmatic dependents) and paged calls, which overlap their neighbours'
    launches and share a workspace, one after the other without a wait: bit for bit what each gives alone."""
    B, types = 3, [SLIDING, FULL, SLIDING, FULL]
    ctx = hd.hybrid_decode_init(hd.Config(layer_types=types, num_q_heads=8, num_kv_heads=2, max_batch=8, max_context=9000,
                                          kv_dtype=hd.HD_KV_FP8_E4M3 if kv == "e4m3" else hd.HD_KV_BF16))
    hd.hybrid_decode_set_step_fusion(ctx, fused)
    rng = synth.generator(140)
    contexts = torch.tensor([8000, 5, 4100], dtype=torch.int32, device="cuda")
    scales = dict(k_scale=synth.kv_scales(rng, 2).cuda(), v_scale=synth.kv_scales(rng, 2).cuda()) if kv == "e4m3" else {}
    layers = []
    for t in types:
        cap = 511 if t == SLIDING else 9001
        kc, vc = (synth.normal_bf16(rng, (B, 2, cap, D)) for _ in range(2))
        if kv == "e4m3":
            kc, vc = synth.e4m3_codes(kc.float()), synth.e4m3_codes(vc.float())
        layers.append([kc.cuda(), vc.cuda()] + [synth.normal_bf16(rng, (B, h, D)).cuda() for h in (8, 2, 2)])
    chunk = PagedCase(141, [(8000, 70), (0, 40)], kv=kv, appended=False)
    single = PagedCase(142, [(8000, 1), (900, 1), (4000, 1)], kv=kv, single=True, appended=False)
    news = {c: [synth.normal_bf16(c.rng, (c.rows, 2, D)).cuda() for _ in range(2)] for c in (chunk, single)}
    bounds = {c: torch.nan_to_num(page_bounds(c)).cuda() for c in (chunk, single)}

    def step(results):
        io, keep = [], []
        for kc, vc, q, k, v in layers:
            kc, vc = kc.clone(), vc.clone()
            out, lse = torch.empty(B, 8, D, dtype=torch.bfloat16, device="cuda"), torch.empty(B, 8, device="cuda")
            io.append(hd.layer_io(q, k, v, hd.kv_cache(kc, vc, **scales), None, out, lse))
            keep += [out, lse, kc, vc]
        results.append(keep)
        return lambda: hd.decode_step(ctx, contexts, io, batch=B)

    def paged(results, case):
        d = case.device()
        k, v = news[case]
        cache, batch = cache_of(hd, d, bounds[case].clone()), case.batch_of(hd, d)
        q_rot, out = torch.empty_like(d["q"]), torch.empty_like(d["q"])
        picked = torch.empty_like(out)
        lse, lse2 = (torch.empty(case.rows, 8, device="cuda") for _ in range(2))
        selected = torch.empty(case.rows, 2, 6, dtype=torch.int32, device="cuda")
        results.append([q_rot, out, lse, picked, lse2, selected, d["k"], d["v"]])

        def call():
            hd.rope_append_paged(ctx, 1, batch, d["q"], k, v, q_rot, cache)
            hd.attn_paged(ctx, 1, batch, q_rot, cache, None, out, lse)
            hd.select_pages(ctx, 1, batch, q_rot, cache, selected)
            hd.attn_selected_pages(ctx, 1, batch, q_rot, cache, selected, None, picked, lse2)
        return call

    def all_of(results):
        return [f for _ in range(3) for f in (step(results), paged(results, chunk), step(results), step(results),
                                              paged(results, single), paged(results, chunk))]

    alone, together = [], []
    for f in all_of(alone):
        f()
        torch.cuda.synchronize()
    calls = all_of(together)
    torch.cuda.synchronize()
    for f in calls:
        f()
    torch.cuda.synchronize()
    assert hd.hybrid_decode_device_errors(ctx) == 0
    for a, b in zip(alone, together):
        for x, y in zip(a, b):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    ctx.close()


@pytest.mark.parametrize("group,spans", [(4, [(700, 1), (4000, 1), (0, 1), (511, 1)]), (4, [(700, 2), (3999, 1), (0, 2), (511, 2)]),
                                         (8, [(700, 1), (4000, 1), (0, 1), (63, 1)]), (1, [(700, 7), (0, 8), (4000, 3), (510, 8)])])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [0, 512])
def test_results_hold_on_both_sides_of_the_choice_of_kernel(hd, orc, group, spans, kv, window):
    """max_tokens x group up to 8 is served by the kernel of few rows, more by the one of chunks."""
    case = PagedCase(150 + group, spans, group=group, kv=kv, window=window)
    ctx, d, sink = context(hd, group, kv=kv), case.device(), sinks(case)
    want = reference_rows(orc, case, sink=sink)
    for max_tokens in (8 // group, 8 // group + 1, 300):
        out, lse = run_attn(hd, ctx, case, d, sink=sink, max_tokens=max_tokens)
        assert hd.hybrid_decode_device_errors(ctx) == 0
        assert_rows(want, out, lse)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_choice_of_blocks_does_not_depend_on_the_bounds(hd, kv):
    case = PagedCase(155, [(3000, 2), (17, 1), (1600, 3)], page=16, kv=kv)
    ctx, d, bounds = context(hd, kv=kv), case.device(), page_bounds(case)
    want = reference_selection(case, bounds, 9, 1, 2)
    for kw in ({}, {"max_context": 3000}, {"max_tokens": 500}, {"max_context": 20000, "max_tokens": 64}):
        selected = torch.full((case.rows, 2, 9), 99, dtype=torch.int32, device="cuda")
        hd.select_pages(ctx, 1, case.batch_of(hd, d, **kw), d["q"], cache_of(hd, d, bounds.cuda()), selected, 1, 2)
        assert np.array_equal(selected.cpu().numpy(), want), kw
    assert hd.hybrid_decode_device_errors(ctx) == 0


def test_queries_are_not_rotated_over_rows_of_others(hd):
    """q_rot at q's own address while q's rows are wider: the rows of the one lie over other rows of the other."""
    case = PagedCase(156, [(5, 3)])
    ctx, d = context(hd), case.device()
    wide = torch.zeros(3, 10, D, dtype=torch.bfloat16, device="cuda")
    q, kv = wide[:, :8], torch.zeros(3, 2, D, dtype=torch.bfloat16, device="cuda")
    q_rot = wide.view(-1)[: 3 * 8 * D].view(3, 8, D)
    batch, cache = case.batch_of(hd, d), cache_of(hd, d)
    for where in (q_rot, wide.view(-1)[D: D + 3 * 8 * D].view(3, 8, D)):
        with pytest.raises(hd.HDError) as e:
            hd.rope_append_paged(ctx, 1, batch, q, kv, kv, where, cache)
        assert e.value.status == 1
    one = case.batch_of(hd, dict(d, offsets=torch.tensor([0, 1], dtype=torch.int32, device="cuda")), num_tokens=1)
    hd.rope_append_paged(ctx, 1, one, q[:1], kv[:1], kv[:1], q_rot[:1], cache)   # one row: in place
    assert hd.hybrid_decode_device_errors(ctx) == 0


@pytest.mark.parametrize("window", [0, 512])
@pytest.mark.parametrize("group", [1, 4, 8])
def test_weights_of_few_rows_keep_their_bits(hd, window, group):
    """Few rows over bf16 pages: beside the output's rounding (2^-8 of it) and the scores' error, only 2^-16 of each weight
    is lost, two roundings of 2^-8 one after the other."""
    case = PagedCase(160 + group, [(700, 1), (63, 1), (4095, 1), (0, 1), (9000, 1)], group=group, window=window, single=True)
    out, _ = run_attn(hd, context(hd, group), case)
    out = out.cpu().double().numpy()
    for r in range(case.rows):
        b, p = case.token(r)
        lo = max(0, p - window + 1) if window else 0
        for h in range(2):
            k, v = (t[torch.from_numpy(case.table[b, lo // 64: p // 64 + 1].astype(np.int64)), h].reshape(-1, D).double().numpy()
                    [lo % 64: lo % 64 + p - lo + 1] for t in (case.k, case.v))
            q = case.q[r, h * group: (h + 1) * group].double().numpy()
            s = q @ k.T / 16
            w = np.exp(s - s.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            want, size = w @ v, w @ np.abs(v)
            score = 256 * 2.0 ** -24 * (np.abs(q) @ np.abs(k).T / 16).max(1, keepdims=True) + 2.0 ** -20
            bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -16 + 2 * score) * size + 1e-30
            excess = np.abs(out[r, h * group: (h + 1) * group] - want) - bound
            assert (excess <= 0).all(), (r, h, excess.max())


def test_strides_of_dimensions_of_one_do_not_matter(hd, orc):
    """One kv head in pages of [slots][heads][dims], one sequence out of a table of many."""
    case = PagedCase(170, [(130, 1)], kv_heads=1, single=True)
    ctx, d = context(hd, kv_heads=1), case.device()
    for name in ("k", "v"):
        d[name] = d[name].as_strided(d[name].shape, (64 * D, D, D, 1))
    d["context"] = torch.tensor([130, 7, 7], dtype=torch.int32, device="cuda")[::3]
    assert d["context"].stride(0) == 3
    out, lse = run_attn(hd, ctx, case, d)
    assert hd.hybrid_decode_device_errors(ctx) == 0
    assert_rows(reference_rows(orc, case), out, lse)
    with pytest.raises(ValueError):   # two heads that way are no pages
        two = torch.zeros(4, 64, 2, D, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
        hd.paged_cache(two, two)
