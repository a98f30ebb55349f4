"""Normed, turned and scored paged calls without a GPU: the descriptors' layout,
the frequencies of scaled angles, refusals, and the visible range of a tile of
rows (paged_rows.cuh), compiled from its source for the host."""
import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from test_paged_host import descriptors
from test_paged_shares_host import CSRC, I32, P, TESTS, host_source

ROOT = os.path.dirname(TESTS)


def test_descriptors_match_the_header(hd, tmp_path):
    structs = {n: getattr(hd, n) for n in ("hd_rope_params", "hd_rope_table", "hd_head_norm", "hd_scoring")}
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "hybrid_decode.h"', "int main(void) {"]
    for name, cls in structs.items():
        lines.append(f'printf("{name} size %zu\\n", sizeof({name}));')
        lines += [f'printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;", "}"]))
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        s, f, v = line.split()
        assert int(v) == (ctypes.sizeof(structs[s]) if f == "size" else getattr(structs[s], f).offset), line


# -------------------------------------------------------------- frequencies --

@pytest.mark.parametrize("rot,theta", [(8, 1e4), (64, 5e6), (128, 1e4), (256, 5e5)])
def test_plain_and_linear_frequencies(hd, rot, theta):
    want = [theta ** (-2 * i / rot) for i in range(rot // 2)]
    f, m = hd.hd_rope_frequencies(rot, theta)
    assert m == 1.0 and np.allclose(f, want, rtol=1e-14)
    f, m = hd.hd_rope_frequencies(rot, theta, hd.HD_ROPE_LINEAR, 4.0)
    assert m == 1.0 and np.allclose(f, np.array(want) / 4, rtol=1e-14)


@pytest.mark.parametrize("rot,theta,original,factor", [(64, 1e4, 4096, 8), (128, 1e4, 16384, 40), (256, 5e5, 8192, 16)])
def test_scaled_frequencies_keep_fast_pairs_and_slow_the_others(hd, rot, theta, original, factor):
    plain = np.array(hd.hd_rope_frequencies(rot, theta)[0])
    turns = original * plain / (2 * math.pi)
    for kind, slow, fast in ((hd.HD_ROPE_RAMP, 1.0, 32.0), (hd.HD_ROPE_BANDS, 1.0, 4.0)):
        f, m = hd.hd_rope_frequencies(rot, theta, kind, factor, original, slow, fast)
        f = np.array(f)
        # The ramp over the pairs' numbers starts and ends at whole numbers around the border pairs.
        step = theta ** (2 / rot) if kind == hd.HD_ROPE_RAMP else 1.0
        assert np.array_equal(f[turns > fast * step], plain[turns > fast * step])
        low = turns < slow / step
        assert np.allclose(f[low], plain[low] / factor, rtol=1e-14)
        assert (f <= plain * (1 + 1e-15)).all() and (f >= plain / factor * (1 - 1e-15)).all()
        assert (np.diff(f / plain) <= 1e-15).all(), "slower pairs are slowed more"
        between = (turns < fast / step) & (turns > slow * step)
        if kind == hd.HD_ROPE_BANDS:
            keep = (turns[between] - slow) / (fast - slow)
            assert np.allclose(f[between], plain[between] * (keep + (1 - keep) / factor), rtol=1e-13)
        assert m == pytest.approx(0.1 * math.log(factor) + 1 if kind == hd.HD_ROPE_RAMP else 1.0, rel=1e-15)
        assert hd.hd_rope_frequencies(rot, theta, kind, factor, original, slow, fast, amplitude=0.75)[1] == 0.75


def test_ramp_that_covers_all_pairs_or_none(hd):
    """A context so short that every pair is slow, so long that every pair is fast, and a ramp of no length."""
    plain = np.array(hd.hd_rope_frequencies(64, 1e4)[0])
    assert np.allclose(hd.hd_rope_frequencies(64, 1e4, hd.HD_ROPE_RAMP, 4.0, 1.0)[0][1:], plain[1:] / 4, rtol=1e-14)
    assert np.array_equal(hd.hd_rope_frequencies(64, 1e4, hd.HD_ROPE_RAMP, 4.0, 1e12)[0], plain)
    f = np.array(hd.hd_rope_frequencies(8, 1e4, hd.HD_ROPE_RAMP, 4.0, 2 * math.pi, 0.999, 1.001)[0])
    assert np.isfinite(f).all() and (f > 0).all()


@pytest.mark.parametrize("bad", [
    dict(rotary_dim=4), dict(rotary_dim=12), dict(rotary_dim=264), dict(rotary_dim=0), dict(theta=1.0), dict(theta=math.inf),
    dict(theta=math.nan), dict(scaling=-1), dict(scaling=4), dict(scaling=1, factor=0.0), dict(scaling=1, factor=-2.0),
    dict(scaling=1, factor=math.nan), dict(scaling=2, factor=4.0), dict(scaling=2, factor=4.0, original_context=4096, slow=2.0, fast=2.0),
    dict(scaling=3, factor=4.0, original_context=4096, slow=0.0, fast=4.0), dict(scaling=2, factor=0.5, original_context=4096),
    dict(amplitude=-1.0), dict(amplitude=math.nan), dict(scaling=3, factor=4.0, original_context=math.inf),
])
def test_frequencies_refuse(hd, bad):
    with pytest.raises(hd.HDError) as e:
        hd.hd_rope_frequencies(**dict(dict(rotary_dim=64), **bad))
    assert e.value.status == 1


def test_null_arguments_are_refused(hd):
    b, c = (ctypes.byref(x) for x in descriptors(hd))
    p = ctypes.byref(hd._rope_params(64, 1e4, 0, 1.0, 0.0, 1.0, 32.0, 0.0))
    f, m = (ctypes.c_double * 128)(), ctypes.c_double()
    assert hd._lib.hd_rope_frequencies(None, f, ctypes.byref(m)) == 1
    assert hd._lib.hd_rope_frequencies(p, None, ctypes.byref(m)) == 1
    assert hd._lib.hd_rope_frequencies(p, f, None) == 1
    assert hd._lib.hd_rope_fill(p, 0, 4096, None) == 1
    assert hd._lib.hd_rope_fill(p, 16, None, None) == 1
    assert hd._lib.hd_rope_fill(p, 16, 4104, None) == 1
    assert hd._lib.norm_rope_append_paged(None, 0, b, None, None, None, 4096, 2048, 4096, 512, 4096, 512, 4096, c, None) == 1
    assert hd._lib.attn_paged_scored(None, 0, b, None, 4096, c, None, None, 4096, 4096, None) == 1
    assert hd._lib.read_paged(None, b, c, 4096, 512, 4096, 512, None) == 1


def test_binding_checks_lists_of_positions(hd):
    hd._check_ints("first", None, 5, torch.device("cpu"))
    good = torch.zeros(5, dtype=torch.int32)
    hd._check_ints("first", good, 5, good.device)
    for bad in (good[:4], good.long(), torch.zeros(10, dtype=torch.int32)[::2], torch.zeros(5, 1, dtype=torch.int32)):
        with pytest.raises(ValueError):
            hd._check_ints("first", bad, 5, good.device)


# ------------------------------------------------------ visible ranges of tiles --

@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    rows = open(os.path.join(CSRC, "paged_rows.cuh")).read()

    def piece(pattern):
        found = re.findall(pattern, rows, re.S)
        assert len(found) == 1, (pattern, len(found))
        return found[0]

    source = host_source().replace("num_kv_heads, group_shift, window; };", "num_kv_heads, group_shift, window; const int32_t *first, *last; };")
    d = tmp_path_factory.mktemp("spans")
    src, so = d / "spans.cpp", d / "spans.so"
    src.write_text("\n".join([
        source, "namespace hd { namespace {", piece(r"struct RowSpan \{.*?\n\};"),
        piece(r"__device__ __forceinline__ RowSpan row_span\(.*?\n\}"),
        piece(r"template <class T>\n__device__ __forceinline__ T scored_tile\(.*?\n\}"),
        piece(r"__device__ __forceinline__ bool span_is_bad\(.*?\n\}"),
        """
extern "C" void tile_of(const PagedAttnArgs *a, int row0, int n, int ctx, int t0, int nt, int shift, int32_t *out) {
    const SeqSpan q{row0, n, ctx};
    const ChunkTile t = scored_tile<ChunkTile>(*a, q, t0, nt, shift);
    out[0] = t.lo; out[1] = t.hi; out[2] = t.u0; out[3] = t.units;
    const RowSpan f = row_span(*a, q, t0), l = row_span(*a, q, t0 + nt - 1);
    out[4] = f.hi; out[5] = l.lo;
    for (int i = 0; i < nt; ++i) {
        const RowSpan s = row_span(*a, q, t0 + i);
        out[6 + 3 * i] = s.lo; out[7 + 3 * i] = s.hi; out[8 + 3 * i] = span_is_bad(s, f, l);
    }
}
}}"""]))
    subprocess.run(["g++", "-std=c++17", "-O1", "-w", "-shared", "-fPIC", "-I", TESTS, "-I", os.path.join(ROOT, "include"), str(src),
                    "-o", str(so)], check=True)
    return ctypes.CDLL(str(so))


class Args(ctypes.Structure):
    _fields_ = [("table", P), ("table_stride", ctypes.c_int64), ("context", P), ("offsets", P), ("batch", I32), ("num_tokens", I32),
                ("max_tokens", I32), ("max_blocks", I32), ("max_context", I32), ("max_position", I32), ("page_shift", I32),
                ("num_pages", I32), ("err", P), ("num_kv_heads", I32), ("group_shift", I32), ("window", I32), ("first", P), ("last", P)]


def tile(lib, n, ctx, t0, nt, window=0, first=None, last=None, shift=5, row0=3):
    arrays = [None if x is None else np.concatenate([np.full(row0, 77), x, np.full(2, -77)]).astype(np.int32) for x in (first, last)]
    a = Args(first=None if arrays[0] is None else arrays[0].ctypes.data, last=None if arrays[1] is None else arrays[1].ctypes.data,
             window=window)
    out = np.zeros(6 + 3 * nt, np.int32)
    lib.tile_of(ctypes.byref(a), row0, n, ctx, t0, nt, shift, out.ctypes.data_as(P))
    return out[:6], out[6:].reshape(nt, 3)


def spans_of(n, ctx, window, first, last):
    """Visible [lo, hi] of every token by the definition."""
    p = ctx + np.arange(n)
    lo = np.maximum(p - window + 1, 0) if window else np.zeros(n, np.int64)
    hi = p.copy()
    if first is not None:
        lo = np.maximum(lo, first)
    if last is not None:
        hi = np.clip(np.minimum(last, ctx + n - 1), -1, None)
    return lo, hi


def check_tile(lib, n, ctx, t0, nt, window, first, last, shift):
    (lo, hi, u0, units, all_hi, all_lo), rows = tile(lib, n, ctx, t0, nt, window, first, last, shift)
    want_lo, want_hi = (x[t0: t0 + nt] for x in spans_of(n, ctx, window, first, last))
    assert np.array_equal(rows[:, 0], want_lo) and np.array_equal(rows[:, 1], want_hi)
    assert units >= 1 and u0 >= 0
    if hi > lo:
        assert 0 <= lo and hi <= ctx + n and u0 << shift <= lo and hi <= (u0 + units) << shift
    for slo, shi, bad in rows:
        if bad or shi < slo:
            continue
        assert lo <= slo and shi < hi, "a row that is served sees nothing outside its tile"
        assert slo <= all_lo and shi >= all_hi, "what every row sees"
    return rows


@pytest.mark.parametrize("seed", range(6))
def test_tiles_of_ascending_spans(lib, seed):
    rng = np.random.default_rng(seed)
    for _ in range(300):
        n, ctx = int(rng.integers(1, 60)), int(rng.choice([0, 3, 500, 70000]))
        t0 = int(rng.integers(0, n))
        nt = int(rng.integers(1, n - t0 + 1))
        top = ctx + n + 40
        first = np.sort(rng.integers(-5, top, n)) if rng.random() < 0.7 else None
        last = np.sort(rng.integers(-5, top, n)) if rng.random() < 0.7 else None
        if rng.random() < 0.2 and last is not None:
            last[-1] = 2 ** 31 - 1
            last[0] = -2 ** 31
        rows = check_tile(lib, n, ctx, t0, nt, int(rng.choice([0, 16, 512])), first, last, int(rng.choice([5, 6, 7])))
        assert not rows[:, 2].any(), "spans that ascend are never flagged"


def test_tiles_of_spans_that_do_not_ascend(lib):
    """Any row that its tile's range or masks would not serve is flagged."""
    rng = np.random.default_rng(9)
    flagged = 0
    for _ in range(2000):
        n, ctx = int(rng.integers(2, 40)), int(rng.choice([0, 200]))
        first, last = rng.integers(0, ctx + n, n), rng.integers(0, ctx + n, n)
        rows = check_tile(lib, n, ctx, 0, n, int(rng.choice([0, 50])), first, last, 5)
        flagged += rows[:, 2].any()
    assert flagged > 1000


def test_a_tile_that_sees_nothing(lib):
    (lo, hi, u0, units, _, _), rows = tile(lib, 4, 100, 0, 4, first=np.array([200, 200, 300, 2 ** 31 - 1]))
    assert units == 1 and u0 == 0 and hi == 0 and lo > 1 << 29 and (rows[:, 1] < rows[:, 0]).all()
