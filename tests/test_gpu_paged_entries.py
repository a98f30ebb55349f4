"""GPU tests of the paged cache's other ways in and out: normed and turned
appends against 64-bit references, tables of angles, and reading entries back.

Tolerances of a normed and rotated value z = y1 c - y2 s (u = 2^-24, half an fp32 step):
  y    the sum of 256 squares, at most 13 roundings deep: 13 u, halved by the root; mean and eps 2 u, rsqrt 4 u;
       three products and a sum (offset + weight): within 2^-20 of itself in all
  c, s each half a step of fp32 (and of the angle's 64-bit rounding, far less): u amplitude
  z    two products and a sum: 3 u of both products
so |z - ref| <= e = 2^-19 (|y1| + |y2|) amplitude, then half a step of the entry's type: 2^-8 of a bf16 value, 2^-4 of an
E4M3 one and at least half its least step 2^-9, in units of the scale, whose reciprocal adds 2^-22.  Values, bounds,
entries read back and everything that stays are compared bit for bit."""
import numpy as np
import pytest
import torch

import synth
from harness import FULL, SLIDING, assert_bits_equal
from paged_harness import D, PagedCase, reference_append
from test_gpu_paged import APPEND_SPANS, cache_of, context

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


TABLES = {
    "halves 64": dict(rotary_dim=64, theta=5e6),
    "halves 256 bands": dict(rotary_dim=256, theta=5e5, scaling=3, factor=16.0, original_context=2048, slow=1.0, fast=4.0),
    "halves 8 linear": dict(rotary_dim=8, theta=1e4, scaling=1, factor=3.0),
    "neighbours 256 ramp": dict(rotary_dim=256, theta=1e4, layout=1, scaling=2, factor=8.0, original_context=1024),
    "neighbours 72": dict(rotary_dim=72, theta=1e4, layout=1, amplitude=1.5),
}
_tables = {}


def table_of(hd, name, positions=20001):
    if (name, positions) not in _tables:
        _tables[name, positions] = hd.rope_table(positions=positions, **TABLES[name])
    return _tables[name, positions]


def angles(hd, name, p):
    """(cos, sin) times the amplitude in 64 bits, of positions p."""
    f, m = hd.hd_rope_frequencies(**{k: v for k, v in TABLES[name].items() if k != "layout"})
    a = np.asarray(p, np.float64)[:, None] * np.array(f)
    return m * np.cos(a), m * np.sin(a), m


def weights(rng, heads, kind):
    if kind is None:
        return None
    w = torch.from_numpy((1 + 0.3 * rng.standard_normal((heads, D) if "heads" in kind else D)).astype(np.float32))
    return w if "f32" in kind else w.to(torch.bfloat16)


def reference(x, w, offset, cs, sn, amp, layout, rot, norm=True, eps=EPS):
    """(z, e) of rows x [rows, heads, 256]: the value and the fp32 error's bound."""
    x = x.double().numpy()
    y = x
    if norm:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if w is not None:
            y = y * (offset + w.double().numpy())
    z, e = y.copy(), 2.0 ** -19 * np.abs(y)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if layout else (slice(0, rot // 2), slice(rot // 2, rot))
    c, s = cs[:, None], sn[:, None]
    z[..., a], z[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    e[..., a] = e[..., b] = 2.0 ** -19 * (np.abs(y[..., a]) + np.abs(y[..., b])) * amp
    return z, e + 1e-37


def assert_bf16(got, z, e, what):
    got = got.double().cpu().numpy()
    over = np.abs(got - z) - (2.0 ** -8 * (np.abs(z) + e) + e)
    assert (over <= 0).all(), f"{what}: {over.max():.3e} over the bound"


def check_append(hd, orc, case, name, *, kind="bf16", offset=0.0, positions=None, norm=True, bounds=True, fused=False, layer=FULL,
                 k_kind="same", eps=EPS):
    rng = case.rng
    rot, layout = (TABLES[name]["rotary_dim"], TABLES[name].get("layout", 0)) if name else (synth.ROPE[layer][0], 0)
    k, v = (synth.normal_bf16(rng, (case.rows, case.kv_heads, D), 3.0) for _ in range(2))
    v[0, 0, 0] = -0.0
    qw, kw = weights(rng, case.q_heads, kind), weights(rng, case.kv_heads, kind if k_kind == "same" else k_kind)
    pos = np.array([case.token(r)[1] for r in range(case.rows)]) if positions is None else np.asarray(positions)
    if name:
        cs, sn, amp = angles(hd, name, pos)
    else:
        cs, sn, amp = *(np.stack(x) for x in zip(*(orc.rope_angles(int(p), *synth.ROPE[layer]) for p in pos))), 1.0
        cs, sn = cs.astype(np.float64), sn.astype(np.float64)
    zq, eq = reference(case.q, qw, offset, cs, sn, amp, layout, rot, norm, eps)
    zk, ek = reference(k, kw, offset, cs, sn, amp, layout, rot, norm, eps)

    d = case.device()
    held = torch.where(case.held.any(1)[:, None, None, None], synth.normal_bf16(rng, (case.pool, case.kv_heads, 2, D)).float(),
                       torch.tensor(float("nan"))).to(torch.bfloat16)
    bounds_d = held.cuda() if bounds else None
    q_rot = torch.full((case.rows + 1, case.q_heads, D), 9.0, dtype=torch.bfloat16, device="cuda")
    q_d, k_d, v_d = case.q.cuda(), k.cuda(), v.cuda()
    if fused:
        q_d, k_d, v_d = torch.cat([q_d, k_d, v_d], 1).split([case.q_heads, case.kv_heads, case.kv_heads], 1)
    ctx = context(hd, case.group, case.kv_heads, case.kv)
    hd.norm_rope_append_paged(
        ctx, layer, case.batch_of(hd, d), q_d, k_d, v_d, q_rot[: case.rows], cache_of(hd, d, bounds_d),
        rope=table_of(hd, name) if name else None, q_weight=None if qw is None else qw.cuda(), k_weight=None if kw is None else kw.cuda(),
        eps=eps, weight_offset=offset, norm=norm,
        positions=None if positions is None else torch.from_numpy(np.asarray(positions, np.int32)).cuda())
    torch.cuda.synchronize()
    assert hd.hybrid_decode_device_errors(ctx) == 0
    assert (q_rot[case.rows:] == 9.0).all()
    assert_bf16(q_rot[: case.rows], zq, eq, "queries")

    _, vp, _, _ = reference_append(orc, case, FULL, None, k, v)
    assert_bits_equal(d["v"], vp, "V pages")
    k_pages, before = d["k"].cpu(), synth.bits(case.k)
    where = [(case.table[b, p // case.page], p % case.page) for b, p in map(case.token, range(case.rows))]
    page, slot = (np.array(x, np.int64) for x in zip(*where))
    rows_k = k_pages[torch.from_numpy(page), :, torch.from_numpy(slot)]
    if case.kv == "e4m3":
        sc = case.k_scale.double().numpy()[None, :, None]
        got = orc.e4m3_to_f64(synth.bits(rows_k)).reshape(zk.shape)
        t, e = np.clip(zk / sc, -448, 448), ek / sc + 2.0 ** -22 * np.abs(zk / sc)
        over = np.abs(got - t) - (np.maximum(2.0 ** -4 * (np.abs(t) + e), 2.0 ** -10) + e)
        assert (over <= 0).all(), f"K codes: {over.max():.3e} over the bound"
        values = got
    else:
        assert_bf16(rows_k, zk, ek, "K entries")
        values = rows_k.double().numpy()
    after = synth.bits(k_pages)
    after[page, :, slot] = before[page, :, slot]
    assert np.array_equal(after, before), "entries of other positions"
    if bounds:
        want = held.double().numpy()
        for r in range(case.rows):
            if slot[r] == 0:
                want[page[r]] = values[r][:, None]
            want[page[r], :, 0] = np.minimum(want[page[r], :, 0], values[r])
            want[page[r], :, 1] = np.maximum(want[page[r], :, 1], values[r])
        touched = np.zeros(case.pool, bool)
        touched[page] = True
        got = bounds_d.double().cpu().numpy()
        assert np.array_equal(got[touched], want[touched]), "bounds of the touched pages"
        assert np.array_equal(synth.bits(bounds_d)[~touched], synth.bits(held)[~touched]), "bounds of the other pages"


@pytest.mark.parametrize("spans", sorted(APPEND_SPANS))
@pytest.mark.parametrize("name", sorted(TABLES))
@pytest.mark.parametrize("kv,page", [("bf16", 16), ("bf16", 256), ("e4m3", 32)])
def test_normed_append(hd, orc, spans, name, kv, page):
    case = PagedCase(301, APPEND_SPANS[spans], page=page, kv=kv, appended=False, single=spans == "single")
    check_append(hd, orc, case, name)


@pytest.mark.parametrize("kind", [None, "bf16", "f32", "bf16 heads", "f32 heads"])
@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_weights(hd, orc, kind, offset):
    case = PagedCase(302, APPEND_SPANS["ragged"], page=16, group=2, kv_heads=3, appended=False, page_gap=64)
    check_append(hd, orc, case, "neighbours 256 ramp", kind=kind, offset=offset, bounds=False, fused=True)
    case = PagedCase(303, APPEND_SPANS["single"], page=64, group=8, kv_heads=1, appended=False, single=True)
    check_append(hd, orc, case, "halves 64", kind=kind, offset=offset)


def test_one_weight_alone(hd, orc):
    for kind, k_kind in (("bf16", None), (None, "f32")):
        check_append(hd, orc, PagedCase(304, APPEND_SPANS["ragged"], appended=False), "halves 64", kind=kind, k_kind=k_kind)


@pytest.mark.parametrize("layer", [SLIDING, FULL])
def test_the_contexts_own_angles(hd, orc, layer):
    check_append(hd, orc, PagedCase(305, APPEND_SPANS["ragged"], appended=False), None, layer=layer, fused=True)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_rotation_without_a_norm(hd, orc, kv):
    check_append(hd, orc, PagedCase(306, APPEND_SPANS["ragged"], kv=kv, appended=False), "neighbours 72", kind=None, norm=False)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_given_positions(hd, orc, kv):
    case = PagedCase(307, APPEND_SPANS["ragged"], kv=kv, appended=False)
    pos = case.rng.integers(0, 20001, case.rows)
    pos[:2] = 0, 20000
    check_append(hd, orc, case, "neighbours 256 ramp", positions=pos)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_small_and_large_rows(hd, orc, kv):
    """Rows of zeros, of 2^-70 (eps alone counts) and of 2^55, and a larger eps."""
    for eps in (1e-6, 0.25):
        case = PagedCase(308, [(5, 40), (1, 3)], page=16, kv=kv, appended=False)
        case.q[0] = 0
        case.q[1] *= 2.0 ** -70
        case.q[2] *= 2.0 ** 55
        check_append(hd, orc, case, "halves 256 bands", eps=eps)


def test_in_place_and_keys_alone(hd, orc):
    case = PagedCase(309, [(5, 40), (100, 3)], appended=False)
    ctx, d = context(hd), case.device()
    k, v = (synth.normal_bf16(case.rng, (case.rows, case.kv_heads, D)).cuda() for _ in range(2))
    q_rot = torch.empty_like(d["q"])
    cache, batch, rope = cache_of(hd, d), case.batch_of(hd, d), table_of(hd, "halves 64")
    hd.norm_rope_append_paged(ctx, 1, batch, d["q"], k, v, q_rot, cache, rope=rope)
    pages = d["k"].clone()
    d["k"].fill_(0)
    hd.norm_rope_append_paged(ctx, 1, batch, None, k, v, None, cache, rope=rope)
    hd.norm_rope_append_paged(ctx, 1, batch, d["q"], k, v, d["q"], cache, rope=rope)
    torch.cuda.synchronize()
    assert torch.equal(d["q"], q_rot)
    for r in range(case.rows):
        b, p = case.token(r)
        at = case.table[b, p // case.page], slice(None), p % case.page
        assert torch.equal(d["k"][at], pages[at])
    assert hd.hybrid_decode_device_errors(ctx) == 0


def test_bad_positions_and_sequences_are_flagged_and_nothing_is_stored(hd, orc):
    case = PagedCase(310, [(5, 4), (100, 3), (60, 1)], appended=False, page=16)
    ctx = context(hd)
    k, v = (synth.normal_bf16(case.rng, (case.rows, case.kv_heads, D)).cuda() for _ in range(2))

    def call(rope, positions=None):
        d = case.device()
        q_rot = torch.full_like(d["q"], 9.0)
        hd.norm_rope_append_paged(ctx, 1, case.batch_of(hd, d), d["q"], k, v, q_rot, cache_of(hd, d), rope=rope, positions=positions)
        torch.cuda.synchronize()
        written = [not torch.equal(d["k"][case.table[b, p // 16], :, p % 16].cpu().view(torch.int16),
                                   case.k[case.table[b, p // 16], :, p % 16].view(torch.int16)) for b, p in map(case.token, range(case.rows))]
        turned = [not bool((q_rot[r] == 9.0).all()) for r in range(case.rows)]
        return written, turned, hd.hybrid_decode_device_errors(ctx)

    # A table of 102 rows: the second sequence reaches position 102.
    ok = [True] * 4 + [False] * 3 + [True]
    assert call(table_of(hd, "halves 64", 102)) == (ok, ok, 4)
    # Given positions below, inside and beyond it.
    pos = torch.tensor([0, -1, 101, 102, 7, 2 ** 31 - 1, -2 ** 31, 5], dtype=torch.int32, device="cuda")
    ok = [True, False, True, False, True, False, False, True]
    assert call(table_of(hd, "halves 64", 102), pos) == (ok, ok, 4)


def test_append_refusals(hd):
    case = PagedCase(311, [(5, 4)], appended=False)
    ctx, d = context(hd), case.device()
    k = torch.zeros(case.rows, case.kv_heads, D, dtype=torch.bfloat16, device="cuda")
    batch, cache, q_rot = case.batch_of(hd, d), cache_of(hd, d), torch.empty_like(d["q"])
    w = torch.ones(D, device="cuda")

    def call(**kw):
        hd.norm_rope_append_paged(ctx, 1, batch, d["q"], k, k, q_rot, cache, **kw)

    for kw in ({"eps": 0.0}, {"eps": -1.0}, {"eps": float("nan")}, {"weight_offset": float("inf")}):
        with pytest.raises(hd.HDError) as e:
            call(**kw)
        assert e.value.status == 1, kw
    for kw in ({"q_weight": w[:128]}, {"q_weight": w.half()}, {"k_weight": w.cpu()}, {"q_weight": w, "k_weight": w.bfloat16()},
               {"q_weight": torch.ones(case.q_heads, D, device="cuda"), "k_weight": w}, {"q_weight": w, "norm": False},
               {"positions": torch.zeros(case.rows + 1, dtype=torch.int32, device="cuda")},
               {"positions": torch.zeros(case.rows, dtype=torch.int64, device="cuda")}):
        with pytest.raises(ValueError):
            call(**kw)
    good = table_of(hd, "halves 64")
    for change in (dict(rotary_dim=12), dict(rotary_dim=0), dict(rotary_dim=512), dict(positions=0), dict(layout=2), dict(table=None),
                   dict(table=good.c.table + 8)):
        c = hd.hd_rope_table(**{f: change.get(f, getattr(good.c, f)) for f, _ in hd.hd_rope_table._fields_})
        with pytest.raises(hd.HDError) as e:
            call(rope=hd.RopeTable(c, good.table))
        assert e.value.status == 1, change
    with pytest.raises(ValueError):
        hd.rope_table(64, 10, layout=2)
    with pytest.raises(ValueError):
        hd.rope_table(64, 10, table=torch.empty(10, 32, 2, device="cuda", dtype=torch.float64))
    call()
    torch.cuda.synchronize()
    assert hd.hybrid_decode_device_errors(ctx) == 0


@pytest.mark.parametrize("name", sorted(TABLES))
def test_tables(hd, name):
    """Every entry half a step of fp32 from the 64-bit value (and a little: the angle's own rounding, the amplitude's product)."""
    t = hd.rope_table(positions=5000, **TABLES[name]).table.double().cpu().numpy()
    cs, sn, amp = angles(hd, name, np.arange(5000))
    for i, want in enumerate((cs, sn)):
        assert (np.abs(t[..., i] - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -38).all()


# -------------------------------------------------------------------- read --

def reference_read(orc, case, t, scale):
    """Bits of every row's entry of pages t."""
    where = [(case.table[b, p // case.page], p % case.page) for b, p in map(case.token, range(case.rows))]
    x = t[torch.tensor([w[0] for w in where]), :, torch.tensor([w[1] for w in where])]
    if case.kv != "e4m3":
        return synth.bits(x)
    return orc.f64_to_bf16(orc.e4m3_to_f64(synth.bits(x)).reshape(x.shape) * scale.double().numpy()[None, :, None])


@pytest.mark.parametrize("spans", sorted(APPEND_SPANS))
@pytest.mark.parametrize("kv,page,kv_heads", [("bf16", 16, 2), ("bf16", 256, 1), ("e4m3", 32, 3), ("e4m3", 128, 4)])
def test_read_back(hd, orc, spans, kv, page, kv_heads):
    case = PagedCase(320, APPEND_SPANS[spans], page=page, kv=kv, kv_heads=kv_heads, single=spans == "single", page_gap=64)
    ctx, d = context(hd, kv_heads=kv_heads, kv=kv), case.device()
    wide = torch.full((case.rows + 2, 2 * kv_heads + 1, D), 9.0, dtype=torch.bfloat16, device="cuda")   # parts of wider rows
    k, v = wide[: case.rows, :kv_heads], wide[: case.rows, kv_heads: 2 * kv_heads]
    hd.read_paged(ctx, case.batch_of(hd, d), cache_of(hd, d), k, v)
    alone = torch.empty(case.rows, kv_heads, D, dtype=torch.bfloat16, device="cuda")
    hd.read_paged(ctx, case.batch_of(hd, d), cache_of(hd, d), v=alone)
    torch.cuda.synchronize()
    assert hd.hybrid_decode_device_errors(ctx) == 0
    assert_bits_equal(k.contiguous(), reference_read(orc, case, case.k, case.k_scale), "keys")
    assert_bits_equal(v.contiguous(), reference_read(orc, case, case.v, case.v_scale), "values")
    assert torch.equal(alone, v)
    assert (wide[case.rows:] == 9.0).all() and (wide[:, 2 * kv_heads:] == 9.0).all()


def test_read_of_every_code(hd, orc):
    """All 254 finite codes with scales whose products need more than fp32's bits."""
    case = PagedCase(321, [(0, 64)], kv="e4m3", page=64)
    codes = torch.arange(256, dtype=torch.uint8).repeat(case.pool * case.kv_heads * 64).view(case.k.shape)
    codes = torch.where((codes & 0x7F) == 0x7F, torch.zeros_like(codes), codes)
    for scale in (1.0 + 2.0 ** -23, 0.333333, 1e-30, 3e35):
        for name in ("k", "v"):
            setattr(case, name, codes.view(case.k.dtype) if case.k.dtype != torch.uint8 else codes.clone())
            setattr(case, name + "_scale", torch.full((case.kv_heads,), scale, dtype=torch.float32))
        ctx, d = context(hd, kv="e4m3"), case.device()
        k = torch.empty(64, case.kv_heads, D, dtype=torch.bfloat16, device="cuda")
        hd.read_paged(ctx, case.batch_of(hd, d), cache_of(hd, d), k)
        torch.cuda.synchronize()
        assert_bits_equal(k, reference_read(orc, case, case.k, case.k_scale), f"scale {scale}")


def test_read_of_bad_sequences_and_pages(hd, orc):
    case = PagedCase(322, [(5, 4), (100, 3), (60, 9), (7, 2)], page=16)
    ctx, d = context(hd), case.device()
    d["context"][1] = -1
    d["table"][2, 64 // 16] = case.pool + 5
    k = torch.full((case.rows + 3, case.kv_heads, D), 9.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, 9.0)
    hd.read_paged(ctx, case.batch_of(hd, d, num_tokens=case.rows + 3), cache_of(hd, d), k, v)
    torch.cuda.synchronize()
    assert hd.hybrid_decode_device_errors(ctx) == 1 | 32
    want = reference_read(orc, case, case.k, None)
    want[4:7] = 0x7FFF
    want[11:16] = 0        # positions 64 .. 68 of the third sequence
    assert_bits_equal(k[: case.rows], want, "keys")
    assert (k[case.rows:] == 9.0).all() and (v[case.rows:] == 9.0).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_read_past_32_bits(hd, kv):
    """Pages whose offsets pass 2^31 elements."""
    pages = 2 ** 31 // (256 * 256) + 300
    shape = (pages, 1, 256, 256)
    ctx = context(hd, kv_heads=1, kv=kv)
    if kv == "e4m3":
        k = torch.zeros(shape, dtype=torch.uint8, device="cuda")
        one = torch.ones(1, device="cuda")
        cache = hd.paged_cache(k, k, one, one)
    else:
        k = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        cache = hd.paged_cache(k, k)
    k[pages - 1, 0, 7] = 0x38 if kv == "e4m3" else 1.0
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    batch = hd.paged_batch(table, torch.tensor([6], dtype=torch.int32, device="cuda"), torch.tensor([0, 3], dtype=torch.int32, device="cuda"),
                           num_tokens=3, max_tokens=3)
    out = torch.full((3, 1, 256), 9.0, dtype=torch.bfloat16, device="cuda")
    hd.read_paged(ctx, batch, cache, out)
    torch.cuda.synchronize()
    assert (out[1] == 1).all() and (out[0] == 0).all() and (out[2] == 0).all()
    assert hd.hybrid_decode_device_errors(ctx) == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_append_past_32_bits(hd, kv):
    """The same entries in the first pages of a pool and behind 2^31 elements."""
    big = 2 ** 31 // (256 * 256) + 4
    ctx = context(hd, kv_heads=1, kv=kv)
    k, v = (torch.zeros(big, 1, 256, D, device="cuda", dtype=torch.uint8 if kv == "e4m3" else torch.bfloat16) for _ in range(2))
    scale = torch.full((1,), 0.01, device="cuda") if kv == "e4m3" else None
    bounds = torch.zeros(big, 1, 2, D, dtype=torch.bfloat16, device="cuda")
    cache = hd.paged_cache(k, v, scale, scale, bounds=bounds)
    rng = synth.generator(5)
    new = [synth.normal_bf16(rng, (300, 1, D)).cuda() for _ in range(2)]
    for at in (0, big - 2):
        batch = hd.paged_batch(torch.tensor([[at, at + 1]], dtype=torch.int32, device="cuda"),
                               torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, 300], dtype=torch.int32, device="cuda"),
                               num_tokens=300, max_tokens=300)
        hd.norm_rope_append_paged(ctx, 1, batch, None, *new, None, cache, rope=table_of(hd, "halves 64"))
    torch.cuda.synchronize()
    assert hd.hybrid_decode_device_errors(ctx) == 0
    for t in (k, v, bounds):
        assert t[0].float().abs().sum() > 0 and torch.equal(t[:2], t[big - 2:])
        assert not t[2: 10].any() and not t[big - 6: big - 2].any()


def test_read_refusals(hd):
    case = PagedCase(323, [(5, 4)])
    ctx, d = context(hd), case.device()
    batch, cache = case.batch_of(hd, d), cache_of(hd, d)
    good = torch.empty(4, case.kv_heads, D, dtype=torch.bfloat16, device="cuda")
    for bad in (good.float(), good[:3], good.cpu(), torch.empty(4, D, case.kv_heads, dtype=torch.bfloat16, device="cuda").transpose(1, 2)):
        with pytest.raises(ValueError):
            hd.read_paged(ctx, batch, cache, bad)
    for k, stride in ((good.data_ptr() + 8, 512), (good.data_ptr(), 504), (good.data_ptr(), 516)):
        assert hd._lib.read_paged(ctx.handle, batch.ref, cache.ref, k, stride, None, 0, None) == 1
    hd.read_paged(ctx, batch, cache)   # nothing to read


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_more_sequences_than_a_block_has_threads(hd, kv):
    """300 sequences of 0 to 2 tokens in one call, on a stream of its own, and in two: the same pages, queries and rows back."""
    ctx = context(hd, kv=kv, max_batch=512)
    rng = synth.generator(6)
    counts = rng.integers(0, 3, 300)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    n = int(offsets[-1])
    contexts = torch.from_numpy(rng.integers(0, 31, 300).astype(np.int32)).cuda()
    table = torch.from_numpy(rng.permutation(600).reshape(300, 2).astype(np.int32)).cuda()
    q, k, v = (synth.normal_bf16(rng, (n, h, D)).cuda() for h in (8, 2, 2))
    scale = torch.full((2,), 0.01, device="cuda") if kv == "e4m3" else None
    rope = table_of(hd, "neighbours 72")
    stream = torch.cuda.Stream()

    def step(parts, stream=None):
        pages = [torch.zeros(600, 2, 16, D, device="cuda").to(torch.float8_e4m3fn if kv == "e4m3" else torch.bfloat16) for _ in range(2)]
        bounds = torch.zeros(600, 2, 2, D, dtype=torch.bfloat16, device="cuda")
        cache = hd.paged_cache(*pages, scale, scale, bounds=bounds)
        q_rot, rk, rv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        torch.cuda.synchronize()
        for a, b in parts:
            r = slice(int(offsets[a]), int(offsets[b]))
            batch = hd.paged_batch(table[a:b], contexts[a:b], torch.from_numpy(offsets[a: b + 1] - offsets[a]).cuda(),
                                   num_tokens=r.stop - r.start, max_tokens=2)
            torch.cuda.synchronize()
            hd.norm_rope_append_paged(ctx, 1, batch, q[r], k[r], v[r], q_rot[r], cache, rope=rope, stream=stream)
            hd.read_paged(ctx, batch, cache, rk[r], rv[r], stream=stream)
        torch.cuda.synchronize()
        assert hd.hybrid_decode_device_errors(ctx) == 0
        return [x.float() for x in (*pages, bounds, q_rot, rk, rv)]

    for a, b in zip(step([(0, 300)], stream), step([(0, 140), (140, 300)])):
        assert torch.equal(a, b)


def test_calls_of_no_tokens(hd):
    case = PagedCase(324, [(5, 0), (90, 0)])
    ctx, d = context(hd), case.device()
    batch, cache = hd.paged_batch(d["table"], d["context"], d["offsets"], num_tokens=0, max_tokens=1), cache_of(hd, d)
    q, k = (torch.empty(0, h, D, dtype=torch.bfloat16, device="cuda") for h in (8, 2))
    hd.norm_rope_append_paged(ctx, 1, batch, q, k, k, q, cache, rope=table_of(hd, "halves 64"))
    hd.read_paged(ctx, batch, cache, k, k)
    hd.attn_paged_scored(ctx, 1, batch, hd.scoring(softcap=30.0), q, cache, None, q, torch.empty(0, 8, device="cuda"))
    torch.cuda.synchronize()
    assert hd.hybrid_decode_device_errors(ctx) == 0


# -------------------------------------------------------- a step of them all --

@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_packed_documents_equal_documents_alone(hd, orc, kv):
    """Three documents packed into one sequence -- positions starting anew, each seeing its own -- give what each gives in a
    sequence of its own: append, attention and the entries read back."""
    sizes = [70, 1, 200]
    rng = synth.generator(77)
    Hq, Hkv, n = 8, 2, sum(sizes)
    ctx = context(hd, kv=kv)
    q, k, v = (synth.normal_bf16(rng, (n, h, D)).cuda() for h in (Hq, Hkv, Hkv))
    qw, kw = (weights(rng, 1, "bf16").cuda() for _ in range(2))
    rope = table_of(hd, "halves 256 bands")
    dtype = torch.float8_e4m3fn if kv == "e4m3" else torch.bfloat16
    scale = torch.full((Hkv,), 3.0 / 448, device="cuda") if kv == "e4m3" else None
    starts = np.concatenate([[0], np.cumsum(sizes)])
    ints = lambda x: torch.tensor(np.asarray(x, np.int32), device="cuda")  # noqa: E731

    def step(spans, table, positions, first):
        pages = [torch.zeros(16, Hkv, 32, D, device="cuda").to(dtype) for _ in range(2)]
        cache = hd.paged_cache(*pages, scale, scale)
        offsets = np.concatenate([[0], np.cumsum(spans)])
        batch = hd.paged_batch(ints(table), ints(np.zeros(len(spans))), ints(offsets), num_tokens=n, max_tokens=max(spans))
        q_rot, out = torch.empty_like(q), torch.empty_like(q)
        lse, rk, rv = torch.empty(n, Hq, device="cuda"), torch.empty_like(k), torch.empty_like(v)
        hd.norm_rope_append_paged(ctx, 1, batch, q, k, v, q_rot, cache, rope=rope, q_weight=qw, k_weight=kw, positions=positions)
        hd.attn_paged_scored(ctx, 1, batch, hd.scoring(softcap=30.0, first=first), q_rot, cache, None, out, lse)
        hd.read_paged(ctx, batch, cache, rk, rv)
        torch.cuda.synchronize()
        assert hd.hybrid_decode_device_errors(ctx) == 0
        return q_rot, out.float(), lse, rk, rv

    packed = step([n], np.arange(9)[None] + 3, ints(np.concatenate([np.arange(s) for s in sizes])), ints(np.repeat(starts[:-1], sizes)))
    apart = step(sizes, np.arange(9 * 3).reshape(3, 9)[:, :7] % 16 * 0 + np.array([[0, 1, 2, 0, 0, 0, 0], [3] * 7, [4, 5, 6, 7, 8, 9, 10]]),
                 None, None)
    for a, b in zip((packed[0], packed[3], packed[4]), (apart[0], apart[3], apart[4])):
        assert torch.equal(a, b)
    # The same sums over the same keys, cut into other tiles: twice the weights' and the output's rounding.
    assert (packed[1] - apart[1]).abs().max() <= 2 * 2.0 ** -8 * 2 * v.abs().max()
    assert (packed[2] - apart[2]).abs().max() <= 2.0 ** -12
    x = v.float() / scale.view(1, -1, 1) if kv == "e4m3" else v
    if kv == "bf16":
        assert torch.equal(packed[4], x)
