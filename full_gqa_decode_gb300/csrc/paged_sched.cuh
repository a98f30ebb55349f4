// Work split of the paged attention kernels.
//
// Items -- a (sequence, tile of its new tokens, kv head) -- differ in length by
// orders of magnitude in one call (a running sequence next to a prompt), and
// only the device knows the lengths.  So the items' key units are laid end to
// end, and CTA i of n takes units [i T / n, (i + 1) T / n) of the T in all:
// every CTA gets the same number, and an item that a border cuts is merged by
// the last of its CTAs (a ticket; nothing waits on another CTA).  Each CTA
// works out T and its start from the lengths alone, one pass over the
// sequences with a block-wide prefix sum.
#pragma once

#include "paged.h"
#include "ptx.cuh"

namespace hd {
namespace {

// A sequence's new tokens; n = 0 when there is nothing to do for it.
struct SeqSpan {
    int row0, n, ctx;
};

// Row range of sequence b, or false (and *bit) when its offsets cannot be used.
__device__ __forceinline__ bool seq_rows(const PagedSeqs &s, int b, int *row0, int *n, int *bit) {
    *row0 = b;
    *n = 1;
    if (s.offsets) {
        const int lo = s.offsets[b], hi = s.offsets[b + 1];
        *row0 = lo;
        *n = 0;
        if (lo < 0 || hi < lo || hi > s.num_tokens) {
            *bit = HD_DEVERR_TOKEN_OFFSETS;
            return false;
        }
        *n = hi - lo;
    }
    return true;
}

// Checked span of sequence b.  *bit: the error of a sequence that cannot be
// served (its span is then empty, *row0 / *rows still name its rows).
__device__ __forceinline__ SeqSpan seq_span(const PagedSeqs &s, int b, int *bit, int *rows = nullptr) {
    SeqSpan q{0, 0, 0};
    *bit = 0;
    int n = 0;
    if (!seq_rows(s, b, &q.row0, &n, bit)) return q;
    if (rows) *rows = n;
    if (n == 0) return q;
    q.ctx = s.context[b];
    if (n > s.max_tokens) *bit = HD_DEVERR_TOKEN_OFFSETS;
    else if (q.ctx < 0) *bit = HD_DEVERR_CONTEXT_NEGATIVE;
    else if (q.ctx > s.max_context || q.ctx > s.max_position - (n - 1)) *bit = HD_DEVERR_CONTEXT_PLAN;
    else if (((q.ctx + n - 1) >> s.page_shift) >= s.max_blocks) *bit = HD_DEVERR_CONTEXT_CAPACITY;
    else q.n = n;
    return q;
}

// The span of the sequence that row r belongs to; n = 0 when there is none or
// it cannot be served (*bit; row0 is past r when no sequence has the row).
__device__ __forceinline__ SeqSpan span_of_row(const PagedSeqs &s, int r, int *bit, int *seq = nullptr) {
    int b = r;
    if (s.offsets) {   // the last sequence that starts at or before r (offsets ascend)
        b = 0;
        for (int hi = s.batch - 1; b < hi;) {
            const int mid = (b + hi + 1) >> 1;
            if (s.offsets[mid] <= r) b = mid;
            else hi = mid - 1;
        }
    }
    if (seq) *seq = b;
    int rows = 0;
    SeqSpan q = seq_span(s, b, bit, &rows);
    if (r < q.row0 || r >= q.row0 + rows) {   // no sequence's row
        q.n = 0;
        q.row0 = 0x7FFFFFFF;
        if (*bit != HD_DEVERR_TOKEN_OFFSETS) *bit = 0;
    }
    return q;
}

// Block-wide prefix sum of 64-bit counts; `tmp`: [33] in shared
// memory.  Returns this thread's exclusive prefix and the total.
__device__ __forceinline__ long long block_prefix(long long x, long long *tmp, long long *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (blockDim.x + 31) >> 5;
    long long v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    if (lane == 31) tmp[warp] = v;
    __syncthreads();
    if (warp == 0) {
        long long w = lane < warps ? tmp[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += t;
        }
        tmp[lane] = w;
    }
    __syncthreads();
    *total = tmp[warps - 1];
    return v - x + (warp ? tmp[warp - 1] : 0);
}

// Which CTA of n holds unit x of T.
__device__ __forceinline__ int cta_of_unit(long long x, long long T, int n) {
    return (int)(((x + 1) * n - 1) / T);
}

}  // namespace
}  // namespace hd
