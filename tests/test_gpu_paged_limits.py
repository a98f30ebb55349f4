"""GPU tests of the paged calls' far ends: scores and biases so large that only the
largest counts, against what is then left of the formula."""
import numpy as np
import pytest
import torch

import synth
from paged_harness import D, U, PagedCase
from scored_harness import Rule, visible
from test_gpu_paged import cache_of, context

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


SPANS = {   # one token, calls of few rows, chunks, and a chunk whose items are cut between CTAs
    "single": [(0, 1), (5, 1), (700, 1), (2047, 1), (9000, 1)],
    "few": [(0, 2), (250, 3), (1000, 1)],
    "chunks": [(0, 150), (300, 90)],
    "cut": [(4000, 70), (5, 20)],
}


def sharp_case(spans, kv, seed=401):
    """Dot products that every kernel sums exactly, whole numbers from -8 to 8 in steps of 2, many of them alike: queries and
    keys of +-1 in eight dims."""
    case = PagedCase(seed, SPANS[spans], kv=kv, single=spans == "single", page=32)

    def signs(shape):
        x = torch.zeros(shape)
        x[..., :8] = torch.from_numpy(np.where(case.rng.random((*shape[:-1], 8)) < 0.5, -1.0, 1.0)).float()
        return x

    case.q = signs(case.q.shape).bfloat16()
    k = signs(case.k.shape)
    if kv == "e4m3":
        case.k_scale = torch.full((case.kv_heads,), 0.25)
        k = synth.e4m3_codes(k / 0.25)
    case.k = torch.where(case.held[:, None, :, None], k.to(case.k.dtype), case.k)
    return case


def run(hd, case, rule):
    ctx, d = context(hd, case.group, case.kv_heads, case.kv), case.device()
    out = torch.full((case.rows, case.q_heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((case.rows, case.q_heads), 7.0, device="cuda")
    hd.attn_paged_scored(ctx, 1, case.batch_of(hd, d), rule.device(hd), d["q"], cache_of(hd, d), None, out, lse)
    torch.cuda.synchronize()
    assert hd.hybrid_decode_device_errors(ctx) == 0
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def seen(orc, case, rule, r, h):
    """(positions, scores, values) that row r sees of kv head h, in 64 bits; scores [group, positions] by the rule."""
    b, _ = case.token(r)
    p, lo, hi = visible(case, rule, r)
    kept = case.__dict__.setdefault("kept", {})
    if (b, h) not in kept:
        pages = case.table[b, : -(-sum(case.spans[b]) // case.page)]
        kept[b, h] = [case.entries(orc, t, s, h, pages) for t, s in ((case.k, case.k_scale), (case.v, case.v_scale))]
    k, v = (x[lo: hi + 1] for x in kept[b, h])
    hs = slice(h * case.group, (h + 1) * case.group)
    x = case.q[r, hs].double().numpy() @ k.T * (rule.scale or 1 / 16)
    if rule.softcap:
        x = rule.softcap * np.tanh(x / rule.softcap)
    if rule.slopes is not None:
        x = x - rule.slopes[hs, None].astype(np.float64) * np.abs(np.arange(lo, hi + 1) - p)
    return np.arange(lo, hi + 1), x, v


def check_largest(orc, case, rule, out, lse, rows, gap):
    """Rows whose largest scores are alike and `gap` above the others, which leave less than 2^-40: the mean of their values.
    out: its own rounding, the weights' to 16 bits, and an fp32 sum of n terms.  lse: the scale's rounding (log2(e)'s and the
    product's), the score's, the bias's, the reference's, the sum's with log2 and the product with ln 2: 8 half steps 2^-24,
    taken as 2^-20; and the product sum's own error, below 2^-6 here."""
    p_round = 2.0 ** -11 if case.kv == "e4m3" else U
    for r in rows:
        for h in range(case.kv_heads):
            at, x, v = seen(orc, case, rule, r, h)
            for i in range(case.group):
                top = x[i].max()
                first = x[i] > top - gap / 2
                assert not ((x[i] > top - gap) & ~first).any(), "the test's own gap"
                n = first.sum()
                want, A = v[first].mean(0), np.abs(v[first]).mean(0)
                row, head = out[r, h * case.group + i], lse[r, h * case.group + i]
                assert np.isfinite(row).all() and np.isfinite(head), f"row {r} head {h * case.group + i}: not finite"
                over = np.abs(row - want) - (U * np.abs(want) + (1.01 * p_round + (n + 8) * 2.0 ** -23) * A + 1e-30)
                assert (over <= 0).all(), f"row {r}: out {over.max():.3e} over its bound"
                assert abs(head - top - np.log(n)) <= 2.0 ** -20 * (1 + abs(top)) + 2.0 ** -6, (r, head, top, n)


@pytest.mark.parametrize("slopes", [False, True])   # slopes of zero: the kernels of biased scores
@pytest.mark.parametrize("scale", [2.0 ** 20, 2.0 ** 24, 2.0 ** 26, 2.0 ** 32])
@pytest.mark.parametrize("spans", sorted(SPANS))
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_large_scales(hd, orc, kv, spans, scale, slopes):
    case = sharp_case(spans, kv)
    rule = Rule(scale=scale, slopes=np.zeros(case.q_heads, np.float32) if slopes else None)
    out, lse = run(hd, case, rule)
    check_largest(orc, case, rule, out, lse, range(0, case.rows, 7), 2 * scale)


@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("scale", [2.0 ** 23, 2.0 ** 28, 2.0 ** 32])
@pytest.mark.parametrize("spans", sorted(SPANS))
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_large_scales_of_any_queries(hd, orc, kv, spans, scale, slopes):
    """Weights are never negative, so an output lies between its column's least and largest visible value, to the weights'
    rounding and its own of the largest magnitude; the largest score is near lse."""
    case = PagedCase(402, SPANS[spans], kv=kv, single=spans == "single", page=32)
    rule = Rule(scale=scale, slopes=np.zeros(case.q_heads, np.float32) if slopes else None)
    out, lse = run(hd, case, rule)
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    for r in range(0, case.rows, 9):
        for h in range(case.kv_heads):
            _, x, v = seen(orc, case, rule, r, h)
            slack = (2.0 ** -7 + 2.0 ** -12) * np.abs(v).max()
            for i in range(case.group):
                row = out[r, h * case.group + i]
                assert (row >= v.min(0) - slack).all() and (row <= v.max(0) + slack).all()
                # 256 half steps of the products' magnitudes, a tenth of the scores' own size here.
                assert abs(lse[r, h * case.group + i] / scale - x[i].max() / scale) < 0.1


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("spans", sorted(SPANS))
def test_the_smallest_scale(hd, orc, kv, spans):
    """Scores of next to nothing: every visible value weighs the same."""
    case = PagedCase(403, SPANS[spans], kv=kv, single=spans == "single", page=32)
    rule = Rule(scale=2.0 ** -32)
    out, lse = run(hd, case, rule)
    check_largest(orc, case, rule, out, lse, range(0, case.rows, 7), 1.0)


STEEP = np.array([1e3, 1e4, 1e5, 1e6, -1e3, -1e5, 300.0, -1e6], np.float32)


@pytest.mark.parametrize("softcap", [0.0, 10.0])
@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("spans", sorted(SPANS))
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_steep_biases(hd, orc, kv, spans, far, softcap):
    """Biases of up to 10^10 in pieces far from their query, where the nearest visible key counts alone (or the farthest); all
    that is visible far behind the query."""
    case = PagedCase(404, SPANS[spans], kv=kv, single=spans == "single", page=32)
    last = None
    if far:
        last = np.concatenate([np.full(n, min(c, 100), np.int64) for c, n in case.spans])
    rule = Rule(softcap=softcap, slopes=STEEP, last=last)
    out, lse = run(hd, case, rule)
    check_largest(orc, case, rule, out, lse, range(0, case.rows, 7), 200.0)
