// Pieces that the paged attention kernels share: the page copy, partial
// weights, the factor of a finished row, and the rows of sequences that cannot
// be served.
#pragma once

#include "paged_sched.cuh"

namespace hd {
namespace {

__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z, int w,
                                            int v) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(smem_u32(bar))
        : "memory");
}

// exp2(x - m) of a partial's maximum x, 0 for a partial that saw no key.
__device__ __forceinline__ float part_weight(float x, float m) { return x == -INFINITY ? 0.f : fast_exp2(x - m); }


// ---- attn_paged_scored ----
__device__ __forceinline__ float fast_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// cap tanh(x / cap) of a score: with e = exp(2 x / cap) it is cap - 2 cap / (1 + e), which keeps an absolute error below
// 2^-21 cap: with u = 2^-24, 2^x (4 u of e, the argument's rounding less) counts 2 u as the slope 2 e / (1 + e)^2 is at most
// half, 1 + e and its reciprocal 3 u of a term of at most 2 cap / (1 + e), the last step u.  e overflows to infinity and
// underflows to 0 where tanh is 1 and -1.
// `z`: x times 2 log2(e) / cap; all else in log2 units.
__device__ __forceinline__ float capped(const PagedAttnArgs &a, float z) {
    return fmaf(-2.f * a.cap, fast_rcp(1.f + fast_exp2(z)), a.cap);
}

__device__ __forceinline__ float min_or_nan(float x, float y) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
// Two binary32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
    float2 r;
    asm("{.reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mul.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d;}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    float2 r;
    asm("{.reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; add.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d;}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    float2 r;
    asm("{.reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7}; fma.rn.f32x2 d, a, b, c;"
        " mov.b64 {%0, %1}, d;}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
    return r;
}
constexpr float kCapReach = 30.f;   // tanh is 1 in binary32 from 2 log2(e) x / cap of 25 on
// capped() of four scores times z, with one reciprocal, of the product of the four 1 + e, and `top` (the cap, or the cap less
// what is to be taken off) in place of the cap.  Three products and the scaling add 4 u of the term to the error: below
// 2^-20 cap in all.  Scores times z must not pass kCapReach, or KEEP keeps the exponents to it.  A NaN among them reaches all
// four.
template <bool KEEP>
__device__ __forceinline__ void capped4(const PagedAttnArgs &a, float z, float top, float (&s)[4]) {
    float2 d[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        d[i] = mul2(make_float2(s[2 * i], s[2 * i + 1]), make_float2(z, z));
        if (KEEP) d[i] = make_float2(min_or_nan(d[i].x, kCapReach), min_or_nan(d[i].y, kCapReach));
        d[i] = add2(make_float2(fast_exp2(d[i].x), fast_exp2(d[i].y)), make_float2(1.f, 1.f));
    }
    const float2 q = mul2(d[0], d[1]);
    const float r = -2.f * a.cap * fast_rcp(q.x * q.y);
    const float2 t = make_float2(r * q.y, r * q.x), c = make_float2(top, top);   // -2 cap over q.x, q.y
    const float2 u = fma2(t, d[1], c), v = fma2(t, d[0], c);
    s[0] = u.x;
    s[1] = u.y;
    s[2] = v.x;
    s[3] = v.y;
}

// Visible positions [lo, hi] of token i of a sequence; none when hi < lo.
struct RowSpan {
    int lo, hi;
};
__device__ __forceinline__ RowSpan row_span(const PagedAttnArgs &a, const SeqSpan &q, int i) {
    const int p = q.ctx + i, r = q.row0 + i;
    RowSpan s{a.window ? max(0, p - a.window + 1) : 0, p};
    if (a.first) s.lo = max(s.lo, a.first[r]);
    if (a.last) s.hi = max(min(a.last[r], q.ctx + q.n - 1), -1);
    return s;
}
// A tile of tokens t0 .. t0 + nt - 1: as both ends of the rows' spans ascend, its first row's lo and its last row's hi hold
// what any of its rows sees.  A tile that sees nothing has one unit outside every page's range, for its rows' zeros.
template <class T>
__device__ __forceinline__ T scored_tile(const PagedAttnArgs &a, const SeqSpan &q, int t0, int nt, int shift) {
    T t;
    t.t0 = t0;
    t.nt = nt;
    t.lo = row_span(a, q, t0).lo;
    t.hi = row_span(a, q, t0 + nt - 1).hi + 1;
    t.u0 = t.lo >> shift;
    t.units = ((t.hi + (1 << shift) - 1) >> shift) - t.u0;
    if (t.hi <= t.lo) {
        t.lo = 0x3FFFFFFF;
        t.hi = t.u0 = 0;
        t.units = 1;
    }
    return t;
}
// Whether row s of a tile whose first and last rows are f and l breaks the ascent (its keys may then lie outside the tile).
__device__ __forceinline__ bool span_is_bad(const RowSpan &s, const RowSpan &f, const RowSpan &l) {
    return s.lo < f.lo || s.lo > l.lo || s.hi < f.hi || s.hi > l.hi;
}

// What a row's unnormalised output is multiplied by -- 1 / l, the E4M3 value
// scale, the sink's share and the gate -- and its lse, from its log2-unit
// maximum m and sum l.  A row that sees no key gives 0 and lse -inf; NaN scores
// stay NaN.
__device__ __forceinline__ float row_factor(const PagedAttnArgs &a, size_t row, int head, float m, float l, float vscale,
                                            float *lse) {
    *lse = l == 0.f ? -INFINITY : (m + fast_log2(l)) * kLn2;
    float f = vscale / l;
    if (a.sink) f *= 1.f / (1.f + fast_exp2((a.sink[head] - *lse) * kLog2e));
    if (a.gate) f *= 1.f / (1.f + fast_exp2(-a.gate[row] * kLog2e));
    return l == 0.f ? 0.f : f;
}

// Rows of a bad sequence: NaN, as the decode calls give.
__device__ __forceinline__ void fill_bad_rows(const PagedAttnArgs &a, int first, int stride) {
    for (int b = first; b < a.seqs.batch; b += stride) {
        int bit, rows = 0;
        const SeqSpan q = seq_span(a.seqs, b, &bit, &rows);
        if (!bit) continue;
        if (threadIdx.x == 0) atomicOr(a.seqs.err, bit);
        const size_t n = (size_t)rows * a.num_q_heads, r0 = (size_t)q.row0 * a.num_q_heads;
        for (size_t i = threadIdx.x; i < n * (kHeadDim / 2); i += blockDim.x)
            reinterpret_cast<uint32_t *>(a.out)[r0 * (kHeadDim / 2) + i] = 0x7FFF7FFFu;
        for (size_t i = threadIdx.x; i < n; i += blockDim.x) a.lse[r0 + i] = __int_as_float(0x7FC00000);
    }
}

}  // namespace
}  // namespace hd
