"""Rules of attn_paged_scored and their 64-bit reference rows, on the CPU.

Tolerances, beside those of paged_harness (u, p and A as there), by the error e_j of a key's score:
  e_j = 256 * 2^-24 * sum_d |q_d k_jd| * scale     the fp32 sum of 256 products
      + 2^-20                                      the exponential, the scaling, the running sums' order
      + 2^-20 * softcap                            the cap's stated error (its slope is at most 1)
      + 2^-21 * (bias_j + bias_top)                the bias in fp32, a product and a sum of it (each half a step,
                                                   2^-24), and the difference to the row's largest score
  out  |gpu - ref| <= u |ref| + f * (p A + 1.1 * (sum_j w_j e_j |v_j| + (sum_j w_j e_j) A))
  lse  |gpu - ref| <= 1.1 * sum_j w_j e_j + 2^-22 (1 + |ref|)
(first order in e_j; the tenth more covers the second, as e_j stays below 0.05 wherever a weight counts.)
"""
from __future__ import annotations

import numpy as np
import torch

from paged_harness import D, U


class Rule:
    def __init__(self, softcap=0.0, scale=0.0, slopes=None, first=None, last=None):
        self.softcap, self.scale, self.slopes, self.first, self.last = softcap, scale, slopes, first, last

    def device(self, hd):
        ints = lambda x: None if x is None else torch.from_numpy(np.asarray(x, np.int32)).cuda()  # noqa: E731
        return hd.scoring(self.softcap, self.scale, None if self.slopes is None else torch.from_numpy(self.slopes).cuda(),
                          ints(self.first), ints(self.last))


def slopes_of(heads, steep=1.0):
    return (steep * 2.0 ** (-8.0 * np.arange(1, heads + 1) / heads)).astype(np.float32)


def documents(case, sizes):
    """first of every row: documents of the given sizes in turn, the first of each sequence begun 7 positions before."""
    out, k = [], 0
    for c, n in case.spans:
        start, end = max(0, c - 7), c + sizes[0] // 2
        for p in range(c, c + n):
            while p >= end:
                start, k = end, k + 1
                end += sizes[k % len(sizes)]
            out.append(start)
    return np.array(out, np.int64)


def prefixes(case, lengths):
    """last of every row: each sequence's first positions see one another."""
    return np.array([max(p, lengths[b % len(lengths)] - 1) if p < lengths[b % len(lengths)] else p
                     for b, (c, n) in enumerate(case.spans) for p in range(c, c + n)], np.int64)


def visible(case, rule, r):
    """(position, lo, hi) of row r."""
    b, p = case.token(r)
    lo = max(0, p - case.window + 1) if case.window else 0
    hi = p
    if rule.first is not None:
        lo = max(lo, int(rule.first[r]))
    if rule.last is not None:
        hi = min(int(rule.last[r]), sum(case.spans[b]) - 1)
    return p, lo, hi


def reference_scored(orc, case, rule, rows=None, sink=None, gate=None):
    """{row: (out [Hq, 256], lse [Hq], tol_out, tol_lse)} in 64 bits."""
    got, keys_of = {}, {}
    p_round = 2.0 ** -11 if case.kv == "e4m3" else U
    scale = rule.scale or 1.0 / 16
    for r in range(case.rows) if rows is None else rows:
        b, _ = case.token(r)
        p, lo, hi = visible(case, rule, r)
        out, tol = np.zeros((case.q_heads, D)), np.full((case.q_heads, D), 1e-30)
        lse, tl = np.full(case.q_heads, -np.inf), np.zeros(case.q_heads)
        if hi >= lo:
            for h in range(case.kv_heads):
                if (b, h) not in keys_of:
                    f0 = max(0, case.spans[b][0] - case.window + 1) // case.page if case.window else 0
                    pages = case.table[b, f0: -(-sum(case.spans[b]) // case.page)]
                    keys_of[b, h] = (f0 * case.page, case.entries(orc, case.k, case.k_scale, h, pages),
                                     case.entries(orc, case.v, case.v_scale, h, pages))
                base, k, v = keys_of[b, h]
                at = np.arange(lo, hi + 1)
                k, v = k[at - base], v[at - base]
                hs = slice(h * case.group, (h + 1) * case.group)
                q = case.q[r, hs].double().numpy()
                s = q @ k.T * scale
                e = 256 * 2.0 ** -24 * (np.abs(q) @ np.abs(k).T * scale) + 2.0 ** -20
                if rule.softcap:
                    s = rule.softcap * np.tanh(s / rule.softcap)
                    e = e + 2.0 ** -20 * rule.softcap
                if rule.slopes is not None:
                    bias = rule.slopes[hs, None].astype(np.float64) * np.abs(at - p)
                    s = s - bias
                    top = np.take_along_axis(np.abs(bias), s.argmax(1)[:, None], 1)
                    e = e + 2.0 ** -21 * (np.abs(bias) + top)
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
                A, we = w @ np.abs(v), w * e
                out[hs] = f * (w @ v)
                tol[hs] = U * np.abs(out[hs]) + f * (p_round * A + 1.1 * (we @ np.abs(v) + we.sum(1, keepdims=True) * A)) + 1e-30
                tl[hs] = 1.1 * we.sum(1) + 2.0 ** -22 * (1 + np.abs(lse[hs]))
        got[r] = (out, lse, tol, tl)
    return got
