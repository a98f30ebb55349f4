"""Inputs and 64-bit references of the paged-cache tests, on the CPU.

Tolerances follow from the roundings (u = 2^-8, half a bf16 step relative to
the value; numpy float64 is exact beside them):
  out  |gpu - ref| <= u |ref| + (p + 2 s) A,  A = sum_j w_j |v_j| with the sink
       and gate factors: the output's own rounding; each weight's rounding to
       the 16-bit type of the second product (p = 2^-8 for bf16 pages, 2^-11 for
       E4M3 pages, whose weights are f16); and the scores' error s in a weight
       and in the sum of weights.
  lse  |gpu - ref| <= s + 2^-22 (1 + |ref|).
  s    the fp32 sum of 256 products of a score, at most 256 half steps 2^-24 of
       sum_d |q_d k_d| / 16 (largest over the row's keys), plus 2^-20 for the
       exponential, the scaling, the running sums' order and the E4M3 path's
       f16 query (2^-25 of its largest value, an eighth of a product's step).
Written entries, selected blocks, bounds and whatever a call must leave alone
are compared bit for bit.
"""
from __future__ import annotations

import numpy as np
import torch

import synth

D = synth.HEAD_DIM
U = 2.0 ** -8


class PagedCase:
    """A pool of pages in random order and sequences with (context, new tokens).  Slots that hold
    nothing yet are NaN, table entries that no call may use are garbage."""

    def __init__(self, seed, spans, *, group=4, kv_heads=2, page=64, kv="bf16", window=0, single=False, spare=3,
                 page_gap=0, appended=True):
        rng = self.rng = np.random.default_rng(seed)
        self.spans, self.group, self.kv_heads, self.page, self.kv, self.window = spans, group, kv_heads, page, kv, window
        self.q_heads = group * kv_heads
        self.batch = len(spans)
        self.single = single
        self.offsets = np.concatenate([[0], np.cumsum([n for _, n in spans])]).astype(np.int32)
        self.rows = int(self.offsets[-1])
        self.max_tokens = max(1, max(n for _, n in spans))
        self.blocks = max(1, max(-(-(c + n) // page) for c, n in spans))
        first = [max(0, c - window + 1) // page if window else 0 for c, _ in spans]
        need = [(b, i) for b, (c, n) in enumerate(spans) for i in range(first[b], -(-(c + n) // page)) if n or c]
        self.pool = len(need) + spare
        order = rng.permutation(self.pool)
        self.table = np.where(rng.random((self.batch, self.blocks)) < 0.5, -7, 2 ** 30).astype(np.int32)
        for i, (b, blk) in enumerate(need):
            self.table[b, blk] = order[i]
        shape = (self.pool, kv_heads, page, D)
        if kv == "e4m3":
            self.k_scale, self.v_scale = synth.kv_scales(rng, kv_heads), synth.kv_scales(rng, kv_heads)
            self.k = synth.e4m3_codes(torch.from_numpy(rng.standard_normal(shape, np.float32)) / self.k_scale.view(-1, 1, 1))
            self.v = synth.e4m3_codes(torch.from_numpy(rng.standard_normal(shape, np.float32)) / self.v_scale.view(-1, 1, 1))
            hole = synth.E4M3_NAN
        else:
            self.k_scale = self.v_scale = None
            self.k, self.v = synth.normal_bf16(rng, shape), synth.normal_bf16(rng, shape)
            hole = float("nan")
        held = torch.zeros(self.pool, page, dtype=torch.bool)
        for b, (c, n) in enumerate(spans):
            lo = max(0, c - window + 1) if window else 0
            for p in range(lo, c + (n if appended else 0)):
                held[self.table[b, p // page], p % page] = True
        for t in (self.k, self.v):
            t.masked_fill_(~held[:, None, :, None], hole)
        self.held = held
        self.q = synth.normal_bf16(rng, (self.rows, self.q_heads, D))
        self.page_gap = page_gap

    # ---- 64-bit values ----
    def entries(self, orc, t, scale, h, pages):
        """float64 [len(pages) * page, 256] of kv head h."""
        x = t[torch.as_tensor(np.asarray(pages, np.int64)), h].reshape(-1, D)
        if self.kv == "e4m3":
            return orc.e4m3_to_f64(x.numpy()) * float(scale[h])
        return x.double().numpy()

    def token(self, r):
        """(sequence, position) of row r."""
        b = int(np.searchsorted(self.offsets, r, side="right") - 1)
        return b, self.spans[b][0] + r - int(self.offsets[b])

    def device(self, dev="cuda"):
        """Device tensors; the pool with `page_gap` elements between pages."""
        out = {}
        for name in ("k", "v"):
            t = getattr(self, name)
            if self.page_gap:
                wide = torch.zeros(self.pool, t[0].numel() + self.page_gap, dtype=t.dtype)
                wide[:, : t[0].numel()] = t.reshape(self.pool, -1)
                wide = wide.to(dev)
                out[name] = wide[:, : t[0].numel()].view(t.shape)
            else:
                out[name] = t.to(dev)
        for name in ("k_scale", "v_scale", "q"):
            t = getattr(self, name)
            out[name] = None if t is None else t.to(dev)
        out["table"] = torch.from_numpy(self.table).to(dev)
        out["context"] = torch.tensor([c for c, _ in self.spans], dtype=torch.int32, device=dev)
        out["offsets"] = None if self.single else torch.from_numpy(self.offsets).to(dev)
        return out

    def batch_of(self, hd, d, **kw):
        kw = dict(dict(num_tokens=self.rows, max_tokens=self.max_tokens), **kw)
        return hd.paged_batch(d["table"], d["context"], d["offsets"], **kw)


def reference_rows(orc, case, rows=None, sink=None, gate=None, selected=None):
    """{row: (out [Hq, 256], lse [Hq], tol_out, tol_lse)} in 64 bits."""
    got = {}
    keys_of = {}
    p_round = 2.0 ** -11 if case.kv == "e4m3" else U
    for r in range(case.rows) if rows is None else rows:
        b, p = case.token(r)
        out, tol = np.zeros((case.q_heads, D)), np.zeros((case.q_heads, D))
        lse, tl = np.full(case.q_heads, -np.inf), np.zeros(case.q_heads)
        lo = max(0, p - case.window + 1) if case.window else 0
        for h in range(case.kv_heads):
            if selected is None:
                at = np.arange(lo, p + 1)
            else:
                blks = [x for x in selected[r, h] if 0 <= x <= p // case.page]
                at = np.concatenate([np.arange(x * case.page, (x + 1) * case.page) for x in blks] or [np.zeros(0, int)])
                at = at[at <= p]
            if len(at) == 0:
                continue
            first = lo // case.page
            if (b, h) not in keys_of:
                f0 = max(0, case.spans[b][0] - case.window + 1) // case.page if case.window else 0
                pages = case.table[b, f0: -(-sum(case.spans[b]) // case.page)]
                keys_of[b, h] = (f0 * case.page, case.entries(orc, case.k, case.k_scale, h, pages),
                                 case.entries(orc, case.v, case.v_scale, h, pages))
            base, k, v = keys_of[b, h]
            k, v = k[at - base], v[at - base]
            hs = slice(h * case.group, (h + 1) * case.group)
            q = case.q[r, hs].double().numpy()
            s = q @ k.T / 16
            m = s.max(1, keepdims=True)
            w = np.exp(s - m)
            total = w.sum(1, keepdims=True)
            w /= total
            lse[hs] = (m + np.log(total))[:, 0]
            f = np.ones((case.group, 1))
            if sink is not None:
                f = f / (1 + np.exp(sink[hs, None].double().numpy() - lse[hs, None]))
            if gate is not None:
                with np.errstate(over="ignore"):
                    f = f / (1 + np.exp(-gate[r, hs, None].double().numpy()))
            es = 256 * 2.0 ** -24 * (np.abs(q) @ np.abs(k).T / 16).max(1, keepdims=True) + 2.0 ** -20
            out[hs] = f * (w @ v)
            tol[hs] = U * np.abs(out[hs]) + f * (p_round + 2 * es) * (w @ np.abs(v)) + 1e-30
            tl[hs] = es[:, 0] + 2.0 ** -22 * (1 + np.abs(lse[hs]))
        got[r] = (out, lse, tol, tl)
    return got


def assert_rows(ref, out, lse):
    out, lse = out.float().cpu().double().numpy(), lse.cpu().double().numpy()
    for r, (o, ls, to, tl) in ref.items():
        assert np.isfinite(out[r]).all(), f"row {r}: non-finite output"
        excess = np.abs(out[r] - o) - to
        assert (excess <= 0).all(), f"row {r}: out {excess.max():.3e} over its bound at {np.unravel_index(excess.argmax(), excess.shape)}"
        none = np.isneginf(ls)
        assert (np.isneginf(lse[r]) == none).all(), f"row {r}: lse of rows without keys"
        d = np.abs(lse[r][~none] - ls[~none]) - tl[~none]
        assert (d <= 0).all(), f"row {r}: lse {d.max():.3e} over its bound"


def reference_append(orc, case, layer_type, q, k, v, bounds=None):
    """Pages, bounds and rotated queries after an append: (k pages, v pages, bounds, q_rot), bit patterns."""
    rot, theta = synth.ROPE[layer_type]
    half = rot // 2
    kp, vp = synth.bits(case.k), synth.bits(case.v)
    bd = None if bounds is None else bounds.float().numpy().copy()
    qr = np.empty((case.rows, case.q_heads, D), np.uint16)

    def turn(x, cs, sn):
        x = x.double().numpy()
        y = x.copy()
        c, s = cs.astype(np.float64), sn.astype(np.float64)
        y[..., :half] = x[..., :half] * c - x[..., half:rot] * s
        y[..., half:rot] = x[..., half:rot] * c + x[..., :half] * s
        return y

    for r in range(case.rows):
        b, p = case.token(r)
        cs, sn = orc.rope_angles(p, rot, theta)
        if q is not None:
            qr[r] = orc.f64_to_bf16(turn(q[r], cs, sn))
        page, slot = case.table[b, p // case.page], p % case.page
        key = turn(k[r], cs, sn)
        for h in range(case.kv_heads):
            if case.kv == "e4m3":
                kp[page, h, slot] = orc.f64_to_e4m3(key[h] / float(case.k_scale[h]))
                vp[page, h, slot] = orc.f64_to_e4m3(v[r, h].double().numpy() / float(case.v_scale[h]))
                stored = orc.e4m3_to_f64(kp[page, h, slot])
            else:
                kp[page, h, slot] = orc.f64_to_bf16(key[h])
                vp[page, h, slot] = synth.bits(v[r, h])
                stored = orc.bf16_to_f64(kp[page, h, slot])
            if bd is not None:
                if slot == 0:
                    bd[page, h] = stored
                bd[page, h, 0] = np.minimum(bd[page, h, 0], stored)
                bd[page, h, 1] = np.maximum(bd[page, h, 1], stored)
    return kp, vp, bd, qr
