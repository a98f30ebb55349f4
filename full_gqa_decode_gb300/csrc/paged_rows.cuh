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
