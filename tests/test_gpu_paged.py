"""GPU tests of the paged-cache calls against 64-bit references: the append
(entries, bounds and queries bit for bit), attention of single tokens and
chunks, the choice of blocks and attention over them, a whole step of them in
order, and what bad inputs on the device do.  Unwritten slots are NaN and
unused table entries garbage, so a wrong read shows."""
import numpy as np
import pytest
import torch

import synth
from harness import FULL, SLIDING, assert_bits_equal
from paged_harness import D, PagedCase, assert_rows, reference_append, reference_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


_contexts = {}


def context(hd, group=4, kv_heads=2, kv="bf16", max_batch=64, max_context=20000, window=512):
    """One sliding (0) and one full (1) layer; kept over the module, as a program would."""
    key = (group, kv_heads, kv, max_batch, max_context, window)
    if key not in _contexts:
        _contexts[key] = hd.hybrid_decode_init(hd.Config(
            layer_types=[SLIDING, FULL], num_q_heads=group * kv_heads, num_kv_heads=kv_heads, max_batch=max_batch,
            max_context=max_context, sliding_window=window,
            kv_dtype=hd.HD_KV_FP8_E4M3 if kv == "e4m3" else hd.HD_KV_BF16))
    return _contexts[key]


def cache_of(hd, d, bounds=None):
    return hd.paged_cache(d["k"], d["v"], d["k_scale"], d["v_scale"], bounds=bounds)


def run_attn(hd, ctx, case, d=None, layer=None, sink=None, gate=None, selected=None, **kw):
    d = d or case.device()
    layer = (0 if case.window else 1) if layer is None else layer
    out = torch.full((case.rows, case.q_heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((case.rows, case.q_heads), 7.0, device="cuda")
    batch, cache = case.batch_of(hd, d, **kw), cache_of(hd, d)
    sink_d, gate_d = (None if t is None else t.cuda() for t in (sink, gate))
    if selected is None:
        hd.attn_paged(ctx, layer, batch, d["q"], cache, sink_d, out, lse, gate=gate_d)
    else:
        hd.attn_selected_pages(ctx, layer, batch, d["q"], cache, selected, sink_d, out, lse, gate=gate_d)
    torch.cuda.synchronize()
    return out, lse


def check_attn(hd, orc, case, rows=None, sink=None, gate=None, ctx=None, **kw):
    ctx = ctx or context(hd, case.group, case.kv_heads, case.kv)
    out, lse = run_attn(hd, ctx, case, sink=sink, gate=gate, **kw)
    assert hd.hybrid_decode_device_errors(ctx) == 0
    assert_rows(reference_rows(orc, case, rows, sink, gate), out, lse)
    return out, lse


def sinks(case, mixed=True):
    return synth.sink_vector(case.rng, ("normal", 2.0 ** 0.5, 0.25 if mixed else 0.0), case.q_heads)


# ------------------------------------------------------------------ append --

APPEND_SPANS = {
    "single": [(0, 1), (1, 1), (15, 1), (16, 1), (63, 1), (64, 1), (700, 1), (4095, 1), (8192, 1)],
    "ragged": [(0, 1), (0, 130), (5, 0), (63, 2), (250, 7), (511, 65), (0, 0), (1000, 33)],
    "one long": [(37, 700)],
}


@pytest.mark.parametrize("spans", sorted(APPEND_SPANS))
@pytest.mark.parametrize("layer_type", [SLIDING, FULL])
@pytest.mark.parametrize("kv,page", [("bf16", 16), ("bf16", 64), ("bf16", 256), ("e4m3", 32), ("e4m3", 128)])
def test_append_is_bit_exact(hd, orc, spans, layer_type, kv, page):
    case = PagedCase(11, APPEND_SPANS[spans], page=page, kv=kv, appended=False, single=spans == "single",
                     page_gap=64 if page == 64 else 0)
    k, v = (synth.normal_bf16(case.rng, (case.rows, case.kv_heads, D)) for _ in range(2))
    k[0, 0, :8] = 0.0      # exact zeros, a negative zero and values beyond E4M3's range
    k[0, 0, 8] = -0.0
    v[0, 0, 0], v[0, 0, 1] = 1e4, -0.0
    held = torch.where(case.held.any(1)[:, None, None, None], synth.normal_bf16(case.rng, (case.pool, case.kv_heads, 2, D)).float(),
                       torch.tensor(float("nan"))).to(torch.bfloat16)
    kp, vp, bd, qr = reference_append(orc, case, layer_type, case.q, k, v, held)
    d = case.device()
    bounds = held.cuda()
    ctx = context(hd, kv=kv)
    q_rot = torch.zeros(case.rows + 2, case.q_heads, D, dtype=torch.bfloat16, device="cuda")
    q_rot[case.rows:] = 9.0
    hd.rope_append_paged(ctx, layer_type, case.batch_of(hd, d), d["q"], k.cuda(), v.cuda(), q_rot[: case.rows],
                         cache_of(hd, d, bounds))
    torch.cuda.synchronize()
    assert hd.hybrid_decode_device_errors(ctx) == 0
    assert_bits_equal(d["k"], kp, "K pages")
    assert_bits_equal(d["v"], vp, "V pages")
    assert_bits_equal(q_rot[: case.rows], qr, "rotated queries")
    assert (q_rot[case.rows:] == 9.0).all()
    touched = np.zeros(case.pool, bool)
    for r in range(case.rows):
        b, p = case.token(r)
        touched[case.table[b, p // page]] = True
    got = bounds.float().cpu().numpy()
    assert np.array_equal(got[touched], bd[touched]), "bounds of the touched pages"
    assert np.array_equal(synth.bits(bounds)[~touched], synth.bits(held)[~touched]), "bounds of the other pages"


@pytest.mark.parametrize("scales", [(0.37, 1.0), (2.0 ** -130, -0.5), (3e38, 2.0 ** -126)])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_append_of_hard_values_is_bit_exact(hd, orc, kv, scales):
    """Entries of every binade from subnormals to the largest, pairs whose rotation cancels, infinities, zeros of
    either sign; scales whose reciprocal is no normal binary32 number."""
    case = PagedCase(14, [(5, 40), (1, 3), (900, 5)], page=16, kv=kv, appended=False)
    rng = case.rng

    def values(heads):
        bits = rng.integers(0, 0x7F80, (case.rows, heads, D)) | rng.integers(0, 2, (case.rows, heads, D)) << 15
        x = torch.from_numpy(bits.astype(np.uint16).view(np.int16)).view(torch.bfloat16)
        half = synth.ROPE[FULL][0] // 2
        for r in range(0, case.rows, 2):   # x1 c - x2 s near zero, at ordinary magnitudes
            cs, sn = orc.rope_angles(case.token(r)[1], 2 * half, synth.ROPE[FULL][1])
            x2 = rng.standard_normal((heads, half)).astype(np.float32)
            x[r, :, half : 2 * half] = torch.from_numpy(x2).bfloat16()
            ratio = (sn / np.where(cs == 0, 1, cs)).astype(np.float64)
            x[r, :, :half] = (x[r, :, half : 2 * half].double() * torch.from_numpy(ratio)).bfloat16()
        x[1, :, :6] = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), 0.0, -0.0], dtype=torch.bfloat16)
        x[3, :, half : half + 2] = 0.0
        x[3, :, :2] = -0.0
        return x

    q, k, v = values(case.q_heads), values(case.kv_heads), values(case.kv_heads)
    if kv == "e4m3":
        case.k_scale = torch.tensor(scales, dtype=torch.float32)
        case.v_scale = torch.tensor(scales[::-1], dtype=torch.float32)
    bounds = torch.zeros(case.pool, case.kv_heads, 2, D, dtype=torch.bfloat16)
    kp, vp, bd, qr = reference_append(orc, case, FULL, q, k, v, bounds)
    d = case.device()
    bounds = bounds.cuda()
    ctx = context(hd, kv=kv)
    q_rot = torch.zeros(case.rows, case.q_heads, D, dtype=torch.bfloat16, device="cuda")
    hd.rope_append_paged(ctx, 1, case.batch_of(hd, d), q.cuda(), k.cuda(), v.cuda(), q_rot, cache_of(hd, d, bounds))
    torch.cuda.synchronize()
    assert hd.hybrid_decode_device_errors(ctx) == 0
    assert_bits_equal(d["k"], kp, "K pages")
    assert_bits_equal(d["v"], vp, "V pages")
    assert_bits_equal(q_rot, qr, "rotated queries")
    assert np.array_equal(bounds.float().cpu().numpy(), bd), "bounds"


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_append_of_parts_of_wider_rows_and_in_place(hd, orc, kv):
    case = PagedCase(12, [(3, 20), (100, 1), (64, 64)], kv=kv, appended=False)
    Hq, Hkv = case.q_heads, case.kv_heads
    row = synth.normal_bf16(case.rng, (case.rows, Hq + 2 * Hkv, D))
    q, k, v = row.split([Hq, Hkv, Hkv], dim=1)
    kp, vp, _, qr = reference_append(orc, case, FULL, q, k, v)
    ctx = context(hd, kv=kv)
    d = case.device()
    wide = row.cuda()
    qd, kd, vd = wide.split([Hq, Hkv, Hkv], dim=1)
    q_rot = torch.empty(case.rows, Hq, D, dtype=torch.bfloat16, device="cuda")
    hd.rope_append_paged(ctx, 1, case.batch_of(hd, d), qd, kd, vd, q_rot, cache_of(hd, d))
    torch.cuda.synchronize()
    assert_bits_equal(d["k"], kp, "K pages")
    assert_bits_equal(d["v"], vp, "V pages")
    assert_bits_equal(q_rot, qr, "rotated queries")
    assert torch.equal(wide.cpu(), row)
    # in place, and keys and values alone
    d2, qc = case.device(), q.contiguous().cuda()
    hd.rope_append_paged(ctx, 1, case.batch_of(hd, d2), qc, kd, vd, qc, cache_of(hd, d2))
    assert_bits_equal(qc, qr, "queries rotated in place")
    d3 = case.device()
    hd.rope_append_paged(ctx, 1, case.batch_of(hd, d3), None, kd, vd, None, cache_of(hd, d3))
    assert_bits_equal(d3["k"], kp, "K pages without queries")
    assert hd.hybrid_decode_device_errors(ctx) == 0


def test_append_equals_rope_append_kv(hd):
    """One token per sequence: the entries are those of the per-sequence cache's call."""
    case = PagedCase(13, [(0, 1), (9, 1), (700, 1), (1023, 1)], appended=False, single=True)
    ctx = context(hd)
    d = case.device()
    k, v = (synth.normal_bf16(case.rng, (case.rows, 2, D)).cuda() for _ in range(2))
    kc, vc = (torch.zeros(4, 2, 20001, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q32 = torch.empty(4, 8, D, device="cuda")
    hd.rope_append_kv(ctx, 1, d["context"], d["q"], k, v, q32, hd.kv_cache(kc, vc))
    q_rot = torch.empty_like(d["q"])
    hd.rope_append_paged(ctx, 1, case.batch_of(hd, d), d["q"], k, v, q_rot, cache_of(hd, d))
    for b, (c, _) in enumerate(case.spans):
        page = case.table[b, c // 64]
        assert torch.equal(d["k"][page, :, c % 64], kc[b, :, c])
        assert torch.equal(d["v"][page, :, c % 64], vc[b, :, c])
    assert ((q_rot.float() - q32).abs() <= 2.0 ** -8 * q32.abs() + 1e-30).all()


# --------------------------------------------------------------- attention --

SINGLE = [(0, 1), (1, 1), (15, 1), (16, 1), (31, 1), (32, 1), (63, 1), (64, 1), (127, 1), (128, 1), (511, 1), (512, 1),
          (700, 1), (1025, 1), (4096, 1), (9001, 1)]


@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("kv,page", [("bf16", 16), ("bf16", 64), ("e4m3", 16), ("e4m3", 128)])
@pytest.mark.parametrize("window", [0, 512])
def test_single_tokens(hd, orc, group, kv, page, window):
    case = PagedCase(20 + group, SINGLE, group=group, page=page, kv=kv, window=window, single=True)
    check_attn(hd, orc, case, sink=sinks(case))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_every_page_size(hd, orc, page, kv):
    spans = [(0, 1), (page - 1, 1), (page, 1), (3 * page + 5, 1), (2500, 1)]
    case = PagedCase(30, spans, page=page, kv=kv, single=True, page_gap=128)
    check_attn(hd, orc, case)


@pytest.mark.parametrize("kv_heads", [1, 3, 4])
def test_other_kv_heads_and_gates(hd, orc, kv_heads):
    case = PagedCase(31, SINGLE, kv_heads=kv_heads, single=True)
    gate = synth.gate_logits(case.rng, case.rows, case.q_heads, specials=True)
    check_attn(hd, orc, case, sink=sinks(case), gate=gate)


CHUNKS = {
    "drafts": [(700, 2), (0, 5), (4095, 1), (63, 7), (512, 3), (5, 0), (1000, 8)],
    "prompts": [(0, 1), (0, 300), (0, 0), (130, 129), (1000, 33), (509, 64)],
    "mixed": [(4000, 1), (0, 257), (2500, 1), (77, 1), (300, 90)],
}


@pytest.mark.parametrize("spans", sorted(CHUNKS))
@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("kv,page", [("bf16", 16), ("bf16", 64), ("e4m3", 32), ("e4m3", 128)])
@pytest.mark.parametrize("window", [0, 512])
def test_chunks(hd, orc, spans, group, kv, page, window):
    case = PagedCase(40 + group, CHUNKS[spans], group=group, page=page, kv=kv, window=window)
    gate = synth.gate_logits(case.rng, case.rows, case.q_heads)
    rows = list(range(0, case.rows, 7)) + [case.rows - 1] if case.rows > 64 else None
    check_attn(hd, orc, case, rows=rows, sink=sinks(case), gate=gate)


@pytest.mark.parametrize("rows", [128, 132])   # at group 4: all of one CTA, and a few of its peer
@pytest.mark.parametrize("kv,page", [("bf16", 16), ("bf16", 32), ("bf16", 128), ("e4m3", 16), ("e4m3", 64)])
@pytest.mark.parametrize("window", [0, 100])
def test_chunks_of_one_ctas_rows_and_just_more(hd, orc, rows, kv, page, window):
    n = rows // 4
    case = PagedCase(60, [(700, n), (0, n - 1), (4000, 1), (129, 5), (63, n)], page=page, kv=kv, window=window)
    check_attn(hd, orc, case, rows=list(range(0, case.rows, 3)) + [case.rows - 1], sink=sinks(case),
               ctx=context(hd, kv=kv, window=window or 512))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_small_window(hd, orc, kv):
    """A window shorter than a page and than a tile of new tokens."""
    case = PagedCase(50, [(0, 40), (5, 1), (100, 70), (300, 9)], window=8, kv=kv)
    check_attn(hd, orc, case, ctx=context(hd, kv=kv, window=8))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_large_scores_and_growing_maxima(hd, orc, kv):
    """Scores that rise by hundreds along the keys: the running maximum moves in every tile."""
    case = PagedCase(51, [(900, 1), (600, 70), (0, 200)], kv=kv)
    case.q = (case.q.float() * 6).to(torch.bfloat16)
    if kv == "bf16":
        ramp = torch.ones(case.pool)
        for b, (c, n) in enumerate(case.spans):
            for blk in range(-(-(c + n) // case.page)):
                ramp[case.table[b, blk]] = 1 + blk / 2
        case.k = (case.k.float() * ramp.view(-1, 1, 1, 1)).to(torch.bfloat16)
    check_attn(hd, orc, case, rows=list(range(0, case.rows, 5)))


def test_long_context_in_many_pieces(hd, orc):
    case = PagedCase(52, [(19990, 1)], single=True)
    check_attn(hd, orc, case, sink=sinks(case))
    case = PagedCase(53, [(19980, 6), (3, 2)])
    check_attn(hd, orc, case)


def test_results_repeat_and_do_not_depend_on_the_bounds(hd):
    case = PagedCase(54, CHUNKS["mixed"])
    ctx, d = context(hd), case.device()
    a = run_attn(hd, ctx, case, d)
    for kw in ({}, {"max_context": 4000}):
        b = run_attn(hd, ctx, case, d, **kw)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_rows_behind_the_last_sequence_stay(hd, orc):
    case = PagedCase(55, [(100, 3), (7, 20)])
    ctx, d = context(hd), case.device()
    n = case.rows + 5
    out = torch.full((n, case.q_heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, case.q_heads), 7.0, device="cuda")
    q = torch.cat([d["q"], torch.full((5, case.q_heads, D), float("nan"), dtype=torch.bfloat16, device="cuda")])
    hd.attn_paged(ctx, 1, case.batch_of(hd, d, num_tokens=n), q, cache_of(hd, d), None, out, lse)
    assert_rows(reference_rows(orc, case), out[: case.rows], lse[: case.rows])
    assert (out[case.rows:] == 7.0).all() and (lse[case.rows:] == 7.0).all()
    # no new token anywhere, and no row at all
    empty = PagedCase(56, [(100, 0), (7, 0)])
    e = empty.device()
    hd.attn_paged(ctx, 1, empty.batch_of(hd, e, num_tokens=n, max_tokens=3), q, cache_of(hd, e), None, out, lse)
    assert (out[case.rows:] == 7.0).all()
    hd.attn_paged(ctx, 1, empty.batch_of(hd, e), e["q"], cache_of(hd, e), None, out[:0], lse[:0])
    assert hd.hybrid_decode_device_errors(ctx) == 0


def many_spans(seed, long_one):
    rng = np.random.default_rng(seed)
    spans = [(int(c), int(n)) for c, n in zip(rng.integers(0, 150, 300), rng.integers(0, 4, 300))]
    if long_one:
        spans[137] = (33, 90)
    return spans


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("long_one", [False, True])
def test_more_sequences_than_a_block_has_threads(hd, orc, kv, long_one):
    """300 sequences of 0 to 3 new tokens, with a chunk among them or without: append, attention, choice of blocks."""
    case = PagedCase(57, many_spans(57, long_one), group=2, page=16, kv=kv, appended=False)
    ctx, d = context(hd, 2, 2, kv, max_batch=300, max_context=300), case.device()
    k, v = (synth.normal_bf16(case.rng, (case.rows, 2, D)) for _ in range(2))
    held = page_bounds(case)
    held = torch.where(torch.isinf(held), torch.tensor(float("nan"), dtype=torch.bfloat16), held)
    kp, vp, bd, _ = reference_append(orc, case, FULL, None, k, v, held)
    bounds = held.cuda()
    batch, cache = case.batch_of(hd, d), cache_of(hd, d, bounds)
    hd.rope_append_paged(ctx, 1, batch, None, k.cuda(), v.cuda(), None, cache)
    assert_bits_equal(d["k"], kp, "K pages")
    assert_bits_equal(d["v"], vp, "V pages")
    case.k, case.v = d["k"].cpu(), d["v"].cpu()
    rows = list(range(0, case.rows, 7)) + [case.rows - 1]
    out, lse = run_attn(hd, ctx, case, d)
    assert_rows(reference_rows(orc, case, rows), out, lse)
    selected = torch.empty(case.rows, 2, 3, dtype=torch.int32, device="cuda")
    hd.select_pages(ctx, 1, batch, d["q"], cache, selected, 1, 1)
    want = reference_selection(case, torch.from_numpy(bd), 3, 1, 1)
    assert np.array_equal(selected.cpu().numpy(), want)
    out, lse = run_attn(hd, ctx, case, d, selected=selected)
    assert_rows(reference_rows(orc, case, rows, selected=want), out, lse)
    assert hd.hybrid_decode_device_errors(ctx) == 0


def test_rows_before_the_first_sequence_stay(hd, orc):
    case = PagedCase(58, [(100, 3), (7, 20), (300, 1)])
    ctx, d = context(hd), case.device()
    n = case.rows + 4
    d["offsets"] = d["offsets"] + 4
    q = torch.cat([torch.full((4, case.q_heads, D), float("nan"), dtype=torch.bfloat16, device="cuda"), d["q"]])
    for max_tokens in (20, 500):
        out = torch.full((n, case.q_heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((n, case.q_heads), 7.0, device="cuda")
        hd.attn_paged(ctx, 1, case.batch_of(hd, d, num_tokens=n, max_tokens=max_tokens), q, cache_of(hd, d), None, out, lse)
        assert_rows(reference_rows(orc, case), out[4:], lse[4:])
        assert (out[:4] == 7.0).all() and (lse[:4] == 7.0).all()
    selected = torch.full((n, 2, 2), 99, dtype=torch.int32, device="cuda")
    bounds = page_bounds(case)
    hd.select_pages(ctx, 1, case.batch_of(hd, d, num_tokens=n), q, cache_of(hd, d, bounds.cuda()), selected)
    assert (selected[:4] == 99).all()
    assert np.array_equal(selected[4:].cpu().numpy(), reference_selection(case, bounds, 2, 1, 1))
    q_rot = torch.full_like(q, 5.0)
    k = torch.zeros(n, 2, D, dtype=torch.bfloat16, device="cuda")
    hd.rope_append_paged(ctx, 1, case.batch_of(hd, d, num_tokens=n), q, k, k, q_rot, cache_of(hd, d))
    assert (q_rot[:4] == 5.0).all() and not (q_rot[4:] == 5.0).any(-1).any(-1).all()
    assert hd.hybrid_decode_device_errors(ctx) == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 70])
def test_sequences_that_share_their_first_pages(hd, orc, kv, n):
    case = PagedCase(59, [(640, n), (640, n), (700, n)], kv=kv)
    case.table[1, :9] = case.table[0, :9]
    case.table[2, :8] = case.table[0, :8]
    check_attn(hd, orc, case)


@pytest.mark.parametrize("n", [1, 70])
def test_offsets_past_32_bits(hd, orc, n):
    """Pages 2^31 + 64 elements apart: the second starts beyond 4 GiB."""
    case = PagedCase(64, [(100, n)], page=64, spare=1, appended=False)
    assert case.table[0, :2].max() >= 1
    gap, H = 2 ** 31 + 64, case.kv_heads
    d = case.device()
    pool = {}
    for name in ("k", "v"):
        flat = torch.empty((case.pool - 1) * gap + H * 64 * D, dtype=torch.bfloat16, device="cuda")
        pool[name] = flat.as_strided((case.pool, H, 64, D), (gap, 64 * D, D, 1))
        pool[name].copy_(d[name])
        d[name] = pool[name]
    ctx = context(hd)
    k, v = (synth.normal_bf16(case.rng, (case.rows, H, D)) for _ in range(2))
    kp, vp, _, _ = reference_append(orc, case, FULL, None, k, v)
    hd.rope_append_paged(ctx, 1, case.batch_of(hd, d), None, k.cuda(), v.cuda(), None, cache_of(hd, d))
    assert_bits_equal(d["k"].contiguous(), kp, "K pages")
    assert_bits_equal(d["v"].contiguous(), vp, "V pages")
    case.k, case.v = d["k"].cpu().contiguous(), d["v"].cpu().contiguous()
    out, lse = run_attn(hd, ctx, case, d)
    assert hd.hybrid_decode_device_errors(ctx) == 0
    assert_rows(reference_rows(orc, case), out, lse)


# ------------------------------------------------------------ page selection --

def page_bounds(case):
    k = case.k.view(torch.float8_e4m3fn).float() if case.kv == "e4m3" else case.k.float()
    dead = ~case.held[:, None, :, None]
    return torch.stack([k.masked_fill(dead, np.inf).amin(2), k.masked_fill(dead, -np.inf).amax(2)], 2).to(torch.bfloat16)


def reference_selection(case, bounds, S, first, last):
    """int32 [rows, Hkv, S] from the definition in 64 bits, ties to the lower block."""
    got = np.full((case.rows, case.kv_heads, S), -1, np.int32)
    bd = bounds.double().numpy()
    for r in range(case.rows):
        b, p = case.token(r)
        n = p // case.page + 1
        for h in range(case.kv_heads):
            q = case.q[r, h * case.group: (h + 1) * case.group].double().numpy()
            x = bd[case.table[b, :n], h]
            score = np.maximum(q[:, None] * x[None, :, 0], q[:, None] * x[None, :, 1]).sum((0, 2))
            score[:first] = np.inf
            score[max(0, n - last):] = np.inf
            pick = np.sort(np.argsort(-score, kind="stable")[:S])
            got[r, h, : len(pick)] = pick
    return got


@pytest.mark.parametrize("group", [1, 4, 8])
@pytest.mark.parametrize("kv,page", [("bf16", 16), ("e4m3", 32)])
@pytest.mark.parametrize("S,first,last", [(1, 0, 0), (5, 1, 1), (33, 2, 3), (128, 0, 1)])
def test_selection_and_attention_over_it(hd, orc, group, kv, page, S, first, last):
    case = PagedCase(60 + group, [(0, 1), (page, 1), (700, 1), (5000, 1), (2047, 3), (17, 2), (9, 0)], group=group, page=page, kv=kv)
    ctx = context(hd, group, kv=kv)
    d = case.device()
    bounds = page_bounds(case)
    selected = torch.full((case.rows + 1, case.kv_heads, S), 99, dtype=torch.int32, device="cuda")
    hd.select_pages(ctx, 1, case.batch_of(hd, d), d["q"], cache_of(hd, d, bounds.cuda()), selected[:-1], first, last)
    want = reference_selection(case, bounds, S, first, last)
    assert np.array_equal(selected[:-1].cpu().numpy(), want)
    assert (selected[-1] == 99).all()
    sink, gate = sinks(case), synth.gate_logits(case.rng, case.rows, case.q_heads)
    out, lse = run_attn(hd, ctx, case, d, sink=sink, gate=gate, selected=selected[:-1])
    assert hd.hybrid_decode_device_errors(ctx) == 0
    assert_rows(reference_rows(orc, case, None, sink, gate, want), out, lse)


def test_selection_of_equal_scores_takes_the_lower_blocks(hd):
    case = PagedCase(70, [(1999, 1)], page=16, single=True)
    bounds = torch.ones(case.pool, 2, 2, D, dtype=torch.bfloat16)
    bounds[case.table[0, 77]] = 2.0
    case.q = case.q.abs()
    d = case.device()
    selected = torch.empty(1, 2, 6, dtype=torch.int32, device="cuda")
    hd.select_pages(context(hd), 1, case.batch_of(hd, d), d["q"], cache_of(hd, d, bounds.cuda()), selected, 1, 1)
    assert selected[0].cpu().tolist() == [[0, 1, 2, 3, 77, 124]] * 2


def test_selection_between_near_equal_scores(hd):
    """Scores that differ by one part in 2^40, summed from terms of mixed sign: fp32 sums cannot rank them."""
    case = PagedCase(71, [(16 * 300 - 1, 1)], page=16, single=True)
    case.q[:] = case.q[0, 0, 0] * 0 + 1.0
    case.q[..., 0] = 2.0 ** -20
    base = synth.normal_bf16(case.rng, (D,))
    bounds = base.expand(case.pool, 2, 2, D).clone()
    order = np.random.default_rng(3).permutation(300)
    for i, blk in enumerate(order):
        bounds[case.table[0, blk], :, :, 0] = 2.0 ** -8 * (1 + (i % 128) / 128) * 2.0 ** (i // 128)
    want = reference_selection(case, bounds, 40, 0, 0)
    d = case.device()
    selected = torch.empty(1, 2, 40, dtype=torch.int32, device="cuda")
    hd.select_pages(context(hd), 1, case.batch_of(hd, d), d["q"], cache_of(hd, d, bounds.cuda()), selected, 0, 0)
    assert np.array_equal(selected.cpu().numpy(), want)


def test_lists_of_the_callers_own(hd, orc):
    """Entries beyond the token's block or negative are skipped; a list without any gives 0 and -inf."""
    case = PagedCase(72, [(100, 1), (300, 1), (40, 1)], page=16, single=True)
    sel = torch.full((3, 2, 4), -1, dtype=torch.int32)
    sel[0, 0, :2] = torch.tensor([2, 6])
    sel[0, 1, :3] = torch.tensor([6, 0, 3])         # any order
    sel[1, 0, :2] = torch.tensor([18, 19])          # 19 is past the token's block 18
    sel[2, 1, 0] = 2
    out, lse = run_attn(hd, context(hd), case, selected=sel.cuda())
    ref = reference_rows(orc, case, selected=sel.numpy())
    assert_rows(ref, out, lse)
    assert (out[1, 4:] == 0).all() and torch.isneginf(lse[1, 4:]).all()
    sink = sinks(case)
    out, lse = run_attn(hd, context(hd), case, selected=sel.cuda(), sink=sink)
    assert (out[1, 4:] == 0).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_all_blocks_selected_is_full_attention(hd, orc, kv):
    case = PagedCase(73, [(100, 1), (777, 1), (0, 1)], kv=kv, single=True)
    ctx, d = context(hd, kv=kv), case.device()
    selected = torch.empty(3, 2, 16, dtype=torch.int32, device="cuda")
    hd.select_pages(ctx, 1, case.batch_of(hd, d), d["q"], cache_of(hd, d, page_bounds(case).cuda()), selected)
    assert_rows(reference_rows(orc, case), *run_attn(hd, ctx, case, d, selected=selected))


# ------------------------------------------------------------ used together --

@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [0, 512])
def test_prompt_then_tokens_equal_one_prompt(hd, orc, kv, window):
    """A prompt in two chunks and four single tokens, appended and attended in order, against the 64-bit
    attention over the finished pages; the same over selected pages for the last token."""
    total, cuts = 640, [0, 300, 636, 637, 638, 639, 640]
    case = PagedCase(80, [(0, total)], page=32, kv=kv, window=0, appended=False)
    layer = 0 if window else 1
    ctx = context(hd, kv=kv)
    k, v = (synth.normal_bf16(case.rng, (total, 2, D)).cuda() for _ in range(2))
    d = case.device()
    bounds = torch.full((case.pool, 2, 2, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    cache = cache_of(hd, d, bounds)
    q_rot = torch.empty_like(d["q"])
    out = torch.empty_like(d["q"])
    lse = torch.empty(total, 8, device="cuda")
    for lo, hi in zip(cuts, cuts[1:]):
        n = hi - lo
        context_d = torch.tensor([lo], dtype=torch.int32, device="cuda")
        offs = None if n == 1 else torch.tensor([0, n], dtype=torch.int32, device="cuda")
        batch = hd.paged_batch(d["table"], context_d, offs, num_tokens=n, max_tokens=n)
        rows = slice(lo, hi)
        hd.rope_append_paged(ctx, layer, batch, d["q"][rows], k[rows], v[rows], q_rot[rows], cache)
        hd.attn_paged(ctx, layer, batch, q_rot[rows], cache, None, out[rows], lse[rows])
    torch.cuda.synchronize()
    assert hd.hybrid_decode_device_errors(ctx) == 0
    case.k, case.v, case.q, case.window = d["k"].cpu(), d["v"].cpu(), q_rot.cpu(), window
    assert_rows(reference_rows(orc, case, list(range(0, total, 37)) + [635, 636, 637, 639]), out, lse)
    case.held[:] = False
    for p in range(total):
        case.held[case.table[0, p // 32], p % 32] = True
    live = case.held.any(1)
    assert np.array_equal(synth.bits(bounds.cpu()[live]), synth.bits(page_bounds(case)[live]))


def test_captured_in_a_graph_and_replayed(hd, orc):
    case = PagedCase(81, [(100, 1), (900, 1), (63, 1)], single=True, appended=False, spare=8)
    ctx, d = context(hd), case.device()
    k, v = (synth.normal_bf16(case.rng, (3, 2, D)).cuda() for _ in range(2))
    bounds = torch.zeros(case.pool, 2, 2, D, dtype=torch.bfloat16, device="cuda")
    cache, batch = cache_of(hd, d, bounds), case.batch_of(hd, d)
    bufs = [torch.empty_like(d["q"]) for _ in range(3)] + [torch.empty(3, 8, device="cuda") for _ in range(2)]
    selected = torch.empty(3, 2, 4, dtype=torch.int32, device="cuda")

    def step():
        hd.rope_append_paged(ctx, 1, batch, d["q"], k, v, bufs[0], cache)
        hd.attn_paged(ctx, 1, batch, bufs[0], cache, None, bufs[1], bufs[3])
        hd.select_pages(ctx, 1, batch, bufs[0], cache, selected)
        hd.attn_selected_pages(ctx, 1, batch, bufs[0], cache, selected, None, bufs[2], bufs[4])

    step()
    torch.cuda.synchronize()
    eager = [t.clone() for t in bufs + [selected, d["k"], d["v"], bounds]]
    for t in bufs + [selected]:
        t.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert hd.hybrid_decode_device_errors(ctx) == 0
    for a, b in zip(eager, bufs + [selected, d["k"], d["v"], bounds]):
        assert np.array_equal(synth.bits(a) if a.dtype == torch.bfloat16 else a.cpu().numpy(),
                              synth.bits(b) if b.dtype == torch.bfloat16 else b.cpu().numpy())


def test_on_another_stream(hd, orc):
    case = PagedCase(82, CHUNKS["drafts"])
    ctx, d = context(hd), case.device()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, lse = run_attn(hd, ctx, case, d)
    assert_rows(reference_rows(orc, case), out, lse)


def test_two_contexts_at_once(hd, orc):
    """Calls of two contexts in flight together on two streams, long ones, again and again."""
    cases = [PagedCase(97, [(19000, 1), (300, 1), (9000, 1)]), PagedCase(98, [(9000, 130), (0, 300)])]
    ctxs = [context(hd), context(hd, max_batch=8)]
    dev, streams = [c.device() for c in cases], [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    first = [run_attn(hd, x, c, d) for x, c, d in zip(ctxs, cases, dev)]
    outs = [[(torch.empty_like(o), torch.empty_like(l)) for o, l in first] for _ in range(6)]
    torch.cuda.synchronize()
    for row in outs:
        for x, c, d, s, (out, lse) in zip(ctxs, cases, dev, streams, row):
            hd.attn_paged(x, 1, c.batch_of(hd, d), d["q"], cache_of(hd, d), None, out, lse, stream=s.cuda_stream)
    torch.cuda.synchronize()
    for c, f in zip(cases, first):
        assert_rows(reference_rows(orc, c, range(0, c.rows, 40)), *f)
    for row in outs:
        assert all(torch.equal(a, b) for got, f in zip(row, first) for a, b in zip(got, f))


# ---------------------------------------------------------------- bad values --

def test_bad_sequences_are_flagged_and_the_rest_served(hd, orc):
    case = PagedCase(90, [(100, 3), (50, 2), (200, 4), (7, 1)])
    ctx, d = context(hd, max_context=1000), case.device()
    for context_values, bit in (([100, -1, 200, 7], 1), ([100, 5000, 200, 7], 4), ([100, 700, 200, 7], 2)):
        d["context"] = torch.tensor(context_values, dtype=torch.int32, device="cuda")
        out, lse = run_attn(hd, ctx, case, d)
        assert hd.hybrid_decode_device_errors(ctx) == bit
        assert torch.isnan(out[3:5].float()).all() and torch.isnan(lse[3:5]).all()
        good = [0, 1, 2, 5, 6, 7, 8, 9]
        assert_rows(reference_rows(orc, case, good), out, lse)
        before = [t.clone() for t in (d["k"], d["v"])]
        k = torch.full((case.rows, 2, D), 3.0, dtype=torch.bfloat16, device="cuda")
        q_rot = torch.full_like(d["q"], 5.0)
        hd.rope_append_paged(ctx, 1, case.batch_of(hd, d), d["q"], k, k, q_rot, cache_of(hd, d))
        assert hd.hybrid_decode_device_errors(ctx) == bit
        assert (q_rot[3:5] == 5.0).all() and not (q_rot[5] == 5.0).all()
        mine = case.table[1, 0]
        assert np.array_equal(synth.bits(before[0][mine]), synth.bits(d["k"][mine]))
        d["k"].copy_(before[0])
        d["v"].copy_(before[1])


def test_bad_single_tokens_are_flagged(hd, orc):
    case = PagedCase(96, [(100, 1), (50, 1), (700, 1)], page=16, single=True)
    ctx, d, bounds = context(hd, max_context=1000), case.device(), page_bounds(case).cuda()
    want = reference_selection(case, bounds.cpu(), 3, 1, 1)
    for value, bit in ((-1, 1), (1001, 4), (900, 2)):
        d["context"] = torch.tensor([100, value, 700], dtype=torch.int32, device="cuda")
        selected = torch.full((3, 2, 3), 99, dtype=torch.int32, device="cuda")
        hd.select_pages(ctx, 1, case.batch_of(hd, d), d["q"], cache_of(hd, d, bounds), selected)
        assert hd.hybrid_decode_device_errors(ctx) == bit
        assert (selected[1] == -1).all() and np.array_equal(selected[::2].cpu().numpy(), want[::2])
        for chosen in (None, selected):
            out, lse = run_attn(hd, ctx, case, d, selected=chosen)
            assert hd.hybrid_decode_device_errors(ctx) == bit
            assert torch.isnan(out[1].float()).all() and torch.isnan(lse[1]).all()
            assert_rows(reference_rows(orc, case, [0, 2], selected=None if chosen is None else want), out, lse)


def test_bad_offsets_are_flagged(hd, orc):
    case = PagedCase(91, [(100, 3), (50, 2), (200, 4)])
    ctx, d = context(hd), case.device()
    for offs, bad in (([0, 3, 2, 9], [1]), ([0, 3, 5, 900], [2]), ([-4, 3, 5, 9], [0])):
        d["offsets"] = torch.tensor(offs, dtype=torch.int32, device="cuda")
        run_attn(hd, ctx, case, d)
        assert hd.hybrid_decode_device_errors(ctx) & 16, offs
    d["offsets"] = torch.from_numpy(case.offsets).cuda()
    out, lse = run_attn(hd, ctx, case, d, max_tokens=3)    # a sequence of 4 above the bound
    assert hd.hybrid_decode_device_errors(ctx) == 16
    assert torch.isnan(out[5:].float()).all()
    assert_rows(reference_rows(orc, case, range(5)), out, lse)


def test_bad_pages_are_flagged(hd, orc):
    case = PagedCase(92, [(100, 1), (200, 1)], single=True)
    ctx, d = context(hd), case.device()
    for page in (-1, case.pool, 2 ** 31 - 1, -2 ** 31):
        table = torch.from_numpy(case.table)
        table[0, 1] = page
        d["table"] = table.cuda()
        out, lse = run_attn(hd, ctx, case, d)
        assert hd.hybrid_decode_device_errors(ctx) == 32
        assert_rows(reference_rows(orc, case, [1]), out, lse)
        before = synth.bits(d["k"])
        k = torch.full((2, 2, D), 3.0, dtype=torch.bfloat16, device="cuda")
        d["context"] = torch.tensor([100, 200 - 1], dtype=torch.int32, device="cuda")
        hd.rope_append_paged(ctx, 1, case.batch_of(hd, d), None, k, k, None, cache_of(hd, d))
        assert hd.hybrid_decode_device_errors(ctx) == 32
        after = synth.bits(d["k"])
        changed = np.unique(np.argwhere(before != after)[:, 0])
        assert list(changed) == [case.table[1, 199 // 64]]
        d = case.device()


def test_lost_copy_times_out_and_the_context_recovers(hd, orc):
    case = PagedCase(93, [(900, 1), (300, 1)], single=True)
    ctx = context(hd)
    hd.hybrid_decode_inject_lost_copy(ctx, 1)
    run_attn(hd, ctx, case)
    assert hd.hybrid_decode_device_errors(ctx) & 8
    hd.hybrid_decode_inject_lost_copy(ctx, -1)
    check_attn(hd, orc, case)


def test_refusals(hd):
    def refused(status, f, *args, **kw):   # 1: invalid argument, 2: unsupported, 3: capacity, 5: state
        with pytest.raises(hd.HDError) as e:
            f(*args, **kw)
        assert e.value.status == status

    case = PagedCase(94, [(100, 1), (300, 1)], page=16, single=True)
    ctx, d = context(hd), case.device()
    batch, bounds = case.batch_of(hd, d), page_bounds(case).cuda()
    cache, plain = cache_of(hd, d, bounds), cache_of(hd, d)
    q, out = d["q"], torch.empty_like(d["q"])
    lse = torch.empty(2, 8, device="cuda")
    sel = torch.empty(2, 2, 4, dtype=torch.int32, device="cuda")
    kv = torch.zeros(2, 2, D, dtype=torch.bfloat16, device="cuda")
    refused(5, hd.select_pages, ctx, 0, batch, q, cache, sel)
    refused(5, hd.attn_selected_pages, ctx, 0, batch, q, cache, sel, None, out, lse)
    refused(1, hd.select_pages, ctx, 1, batch, q, plain, sel)
    refused(1, hd.select_pages, ctx, 1, batch, q, cache, sel, 3, 2)
    refused(1, hd.select_pages, ctx, 1, batch, q, cache, sel, -1, 2)
    refused(1, hd.attn_paged, ctx, 2, batch, q, cache, None, out, lse)
    refused(1, hd.rope_append_paged, ctx, 1, batch, None, torch.zeros(2, 4 + 2 * D, dtype=torch.bfloat16,
            device="cuda")[:, :2 * D].view(2, 2, D), kv, None, cache)
    odd = torch.zeros(2 * 2 * D + 8, dtype=torch.bfloat16, device="cuda")[4:4 + 2 * 2 * D].view(2, 2, D)
    refused(1, hd.rope_append_paged, ctx, 1, batch, None, odd, kv, None, cache)
    small = context(hd, max_batch=1, max_context=16)
    refused(3, hd.attn_paged, small, 1, batch, q, cache, None, out, lse)
    many = PagedCase(95, [(0, 64)] * 1, page=16)
    m = many.device()
    wide = torch.empty(4096, 8, D, dtype=torch.bfloat16, device="cuda")
    refused(3, hd.select_pages, context(hd, max_batch=1, max_context=262144), 1,
            hd.paged_batch(torch.zeros(1, 16384, dtype=torch.int32, device="cuda"), m["context"], m["offsets"],
                           num_tokens=4096, max_tokens=4096),
            wide, cache_of(hd, m, page_bounds(many).cuda()), torch.empty(4096, 2, 4, dtype=torch.int32, device="cuda"))
    ctx8 = hd.hybrid_decode_init(hd.Config(layer_types=[FULL], num_q_heads=8, num_kv_heads=2, max_batch=2, max_context=400,
                                           sliding_window=64, rotary_dim_full=36))
    refused(2, hd.rope_append_paged, ctx8, 0, batch, None, kv, kv, None, cache)
    ctx8.close()
    for bad in (dict(q=q, q_rot=None), dict(q=None, q_rot=out)):
        with pytest.raises(ValueError):
            hd.rope_append_paged(ctx, 1, batch, bad["q"], kv, kv, bad["q_rot"], cache)
    assert hd.hybrid_decode_device_errors(ctx) == 0
