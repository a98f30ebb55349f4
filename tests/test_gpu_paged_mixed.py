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
