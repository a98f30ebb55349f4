"""GPU tests of the normed append's edges and of what it stores, and of its tables
of angles.  Tolerances as in test_gpu_paged_entries.py."""
import numpy as np
import pytest
import torch

import synth
from harness import FULL, assert_bits_equal
from paged_harness import D, PagedCase, reference_append
from test_gpu_paged import cache_of, context
from test_gpu_paged_entries import APPEND_SPANS, angles, check_append, reference, reference_read, table_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_bounds_of_pages_whose_rows_are_not_all_stored(hd, kv):
    """Rows whose given position is not in the table stay out of the bounds; a page that gets no row keeps its bounds to the
    bit, and one whose first slot is not written keeps what it had among them."""
    case = PagedCase(501, [(0, 40), (5, 8), (20, 3), (16, 16)], kv=kv, page=16, appended=False)
    ctx, d = context(hd, kv=kv), case.device()
    k, v = (synth.normal_bf16(case.rng, (case.rows, case.kv_heads, D), 0.5).cuda() for _ in range(2))
    held = synth.normal_bf16(case.rng, (case.pool, case.kv_heads, 2, D))
    held[:, :, 0] -= 0.5
    held[:, :, 1] += 0.5
    bad = np.zeros(case.rows, bool)
    bad[:16] = True                  # all of a page that the call starts
    bad[[16, 19]] = True             # the first slot of one, and another
    bad[33:40] = True                # all but the first slot
    bad[40:48] = True                # all of a page that has entries
    bad[51 + 1: 51 + 16] = True      # one row in a warp, none in the others
    held[case.table[1, 0]] = float("nan")
    held[case.table[0, 0], 0, 0, :2] = float("inf")
    pos = np.where(bad, 102, np.arange(case.rows) % 102)
    bounds = held.cuda()
    hd.norm_rope_append_paged(ctx, 1, case.batch_of(hd, d), None, k, v, None, cache_of(hd, d, bounds), rope=table_of(hd, "halves 64", 102),
                              positions=torch.from_numpy(pos.astype(np.int32)).cuda())
    torch.cuda.synchronize()
    assert hd.hybrid_decode_device_errors(ctx) == 4
    pages = d["k"].cpu()
    if kv == "e4m3":
        pages = pages.view(torch.float8_e4m3fn)
    want = held.float()
    for r in np.flatnonzero(~bad):   # in order: a page's first slot comes first
        b, p = case.token(r)
        page, x = case.table[b, p // 16], pages[case.table[b, p // 16], :, p % 16].float()
        if p % 16 == 0:
            want[page] = x[:, None]
        want[page, :, 0], want[page, :, 1] = torch.minimum(want[page, :, 0], x), torch.maximum(want[page, :, 1], x)
    assert_bits_equal(bounds, synth.bits(want.to(torch.bfloat16)), "bounds")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_heads_of_the_largest_values(hd, orc, kv):
    """Every value of a head +-2^60: its squares sum to 2^128, which fp32 does not hold."""
    case = PagedCase(502, [(5, 40), (1, 3)], page=16, kv=kv, appended=False)
    signs = lambda shape: torch.from_numpy(np.where(case.rng.random(shape) < 0.5, -1.0, 1.0)).to(torch.bfloat16)  # noqa: E731
    case.q[:4] = signs(case.q[:4].shape) * 2.0 ** 60
    case.q[4] = signs(case.q[4].shape) * 1.9921875 * 2.0 ** 59
    check_append(hd, orc, case, "halves 256 bands")
    check_append(hd, orc, case, "neighbours 72", kind=None)


@pytest.mark.parametrize("scale", [2.0 ** -130, 2.0 ** -149, 2.0 ** -127, 3e38])
@pytest.mark.parametrize("name", ["halves 64", "neighbours 72"])
def test_scales_without_a_reciprocal(hd, orc, name, scale):
    """K scales whose reciprocal is infinite or subnormal: zeros stay zeros, what is beyond 448 saturates, and values of the
    scale's own size are coded as their quotients."""
    case = PagedCase(503, [(5, 40), (1, 3)], kv="e4m3", page=16, appended=False)
    case.k_scale = torch.full((case.kv_heads,), scale, dtype=torch.float32)
    rng, ctx, d = case.rng, context(hd, kv="e4m3"), case.device()
    k = torch.from_numpy(rng.standard_normal((case.rows, case.kv_heads, D)) * min(100 * scale, 2.0 ** 125))
    k[0] = 0.0
    k[1] = torch.from_numpy(np.where(rng.random(k[1].shape) < 0.5, -1.0, 1.0)) * 2.0 ** 100   # beyond 448, but for 3e38: zero
    k[2, :, ::3] = 0.0
    k = k.to(torch.bfloat16)
    hd.norm_rope_append_paged(ctx, 1, case.batch_of(hd, d), None, k.cuda(), k.cuda(), None, cache_of(hd, d), rope=table_of(hd, name),
                              norm=False)
    torch.cuda.synchronize()
    assert hd.hybrid_decode_device_errors(ctx) == 0
    at = [case.token(r) for r in range(case.rows)]
    cs, sn, amp = angles(hd, name, [p for _, p in at])
    rot, layout = (64, 0) if name == "halves 64" else (72, 1)
    z, _ = reference(k, None, 0.0, cs, sn, amp, layout, rot, norm=False)
    rows = torch.stack([d["k"][case.table[b, p // 16], :, p % 16] for b, p in at])
    got = orc.e4m3_to_f64(synth.bits(rows)).reshape(z.shape)
    sc = float(case.k_scale[0])
    # e: the rotation's fp32 error, and subnormal products and sums (three half steps of 2^-149) over the scale; the
    # quotient's half step; then half a code's step.
    a = np.abs(z)
    other = np.zeros_like(a)
    x = np.abs(k.double().numpy())
    other[..., :rot] = np.repeat(x[..., :rot].max(-1, keepdims=True), rot, -1) * amp
    e = 2.0 ** -19 * (a + other) / sc + 1.5 * 2.0 ** -149 / sc * (a > 0) + 2.0 ** -22 * np.minimum(a / sc, 1e6)
    t = np.clip(z / sc, -448, 448)
    over = np.abs(got - t) - (np.maximum(2.0 ** -4 * (np.abs(t) + e), 2.0 ** -10) + e)
    assert np.isfinite(got).all() and (got[0] == 0).all()
    assert (over <= 0).all(), f"{over.max():.3e} over the bound"


@pytest.mark.parametrize("spans", ["ragged", "single"])
def test_e4m3_entries_read_back_after_a_normed_append(hd, orc, spans):
    """The rows that come back are the stored codes times their scale, rounded once: for values the codes of the given rows,
    for keys codes within a normed and rotated key's bound (check_append)."""
    case = PagedCase(504, APPEND_SPANS[spans], kv="e4m3", page=32, appended=False, single=spans == "single")
    ctx, d = context(hd, kv="e4m3"), case.device()
    k, v = (synth.normal_bf16(case.rng, (case.rows, case.kv_heads, D), 3.0) for _ in range(2))
    batch, cache = case.batch_of(hd, d), cache_of(hd, d)
    hd.norm_rope_append_paged(ctx, 1, batch, None, k.cuda(), v.cuda(), None, cache, rope=table_of(hd, "halves 256 bands"))
    rk, rv = torch.empty_like(k, device="cuda"), torch.empty_like(v, device="cuda")
    hd.read_paged(ctx, batch, cache, rk, rv)
    torch.cuda.synchronize()
    assert hd.hybrid_decode_device_errors(ctx) == 0
    _, vp, _, _ = reference_append(orc, case, FULL, None, k, v)
    assert_bits_equal(rv, reference_read(orc, case, torch.from_numpy(vp), case.v_scale), "values")
    assert_bits_equal(rk, reference_read(orc, case, d["k"].cpu(), case.k_scale), "keys")
    cs, sn, amp = angles(hd, "halves 256 bands", [case.token(r)[1] for r in range(case.rows)])
    z, e = reference(k, None, 0.0, cs, sn, amp, 0, 256)
    sc = case.k_scale.double().numpy()[None, :, None]
    t, e = np.clip(z / sc, -448, 448), e / sc + 2.0 ** -22 * np.abs(z / sc)
    got = rk.double().cpu().numpy() / sc
    over = np.abs(got - t) - (np.maximum(2.0 ** -4 * (np.abs(t) + e), 2.0 ** -10) + e + 2.0 ** -8 * np.abs(got))
    assert (over <= 0).all(), f"{over.max():.3e} over the bound"


def test_a_table_filled_on_a_stream_of_its_own(hd):
    """Its memory may have been something else's, which the current stream is still to write."""
    shape, stream = (5000, 32, 2), torch.cuda.Stream()
    want = hd.rope_table(64, 5000, theta=1e4).table.clone()
    torch.cuda.synchronize()
    for given in (stream, stream.cuda_stream):
        torch.cuda._sleep(200_000_000)
        torch.empty(shape, device="cuda").fill_(7.0)   # freed, and still to be filled
        got = hd.rope_table(64, 5000, theta=1e4, stream=given).table
        torch.cuda.synchronize()
        assert torch.equal(got, want)
