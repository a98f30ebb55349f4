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

// Row range of sequence b, or false (and *bit) when its offsets cannot be used: then the rows among them that exist.
__device__ __forceinline__ bool seq_rows(const PagedSeqs &s, int b, int *row0, int *n, int *bit) {
    *row0 = b;
    *n = 1;
    if (s.offsets) {
        const int lo = s.offsets[b], hi = s.offsets[b + 1];
        *row0 = lo;
        *n = 0;
        if (lo < 0 || hi < lo || hi > s.num_tokens) {
            *bit = HD_DEVERR_TOKEN_OFFSETS;
            *row0 = max(lo, 0);
            *n = max(min(hi, s.num_tokens) - *row0, 0);
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
    const bool usable = seq_rows(s, b, &q.row0, &n, bit);
    if (rows) *rows = n;
    if (!usable || n == 0) return q;
    q.ctx = s.context[b];
    if (n > s.max_tokens) *bit = HD_DEVERR_TOKEN_OFFSETS;
    else if (q.ctx < 0) *bit = HD_DEVERR_CONTEXT_NEGATIVE;
    else if (q.ctx > s.max_context || q.ctx > s.max_position - (n - 1)) *bit = HD_DEVERR_CONTEXT_PLAN;
    else if (((q.ctx + n - 1) >> s.page_shift) >= s.max_blocks) *bit = HD_DEVERR_CONTEXT_CAPACITY;
    else q.n = n;
    return q;
}

// The span of the sequence that row r belongs to (the whole warp asks for the
// same row); n = 0 when there is none or it cannot be served (*bit; row0 is past
// r when no sequence has the row).  Offsets ascend: each round the lanes probe
// 32 of them, so 1024 sequences take two loads in a row.
__device__ __forceinline__ SeqSpan span_of_row(const PagedSeqs &s, int r, int *bit, int *seq = nullptr) {
    int b = r;
    if (s.offsets) {
        const int lane = threadIdx.x & 31;
        int lo = 0, n = s.batch;   // the last sequence that starts at or before r is in [lo, lo + n)
        while (n > 1) {
            const int step = (n + 31) >> 5, at = lo + lane * step;
            const bool starts = lane * step < n && s.offsets[at] <= r;
            const int k = 31 - __clz(__ballot_sync(0xffffffffu, starts) | 1u);
            n = min(step, n - k * step);
            lo += k * step;
        }
        b = lo;
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
// memory, which every thread reads last: callers owe a barrier before `tmp` is
// written again.  Returns this thread's exclusive prefix and the total.
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

// Launched as a programmatic dependent of the previous kernel in the stream: set-up that touches no global memory
// runs while that one drains, and everything else behind this wait.
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;"); }

// Where a worker's share of the call's units starts: sequence, tile of its new
// tokens, kv head, and units of that item already passed.
struct Start {
    int b, tile, h, off;
};

constexpr int kFewTiles = 4;   // of a sequence, that one lane counts

// Share `who` of at most `workers` over all units of the call: its first unit
// x0, its end x1 (x0 >= x1: none), the number of shares n and the total T.
// Shares have at least `least` units, unless `items` (about as many as there
// are) asks for more shares.  With `snap`, in a call of at most `mean` units a
// share on average, a border inside an item of at most `snap` units moves to the
// nearer end of the item: merging a cut item costs more than the imbalance.  The
// start may then lie at its item's end (off = its units).  All threads of the
// block call it; `tmp`: 33 64-bit words, `at`: 5 words of shared memory.
// *bad: some sequence cannot be served.
//   tiles(n)      tiles of n new tokens
//   units(q, i)   units of one kv head of tile i of span q
template <class Tiles, class Units>
__device__ __forceinline__ Start find_share(const PagedSeqs &s, int num_kv_heads, int who, int workers, int least,
                                            int items, int snap, int mean, long long *tmp, int *at, long long *x0, long long *x1, long long *T, int *n,
                                            int *bad, Tiles tiles, Units units) {
    const int lane = threadIdx.x & 31;
    // Up to 32 sequences every warp works it out by itself; above, the block together.
    const bool by_warp = s.batch <= 32;
    const int who_am = by_warp ? lane : (int)threadIdx.x, of = by_warp ? 32 : (int)blockDim.x;
    const int per = (s.batch + of - 1) / of;
    const int b_lo = min(who_am * per, s.batch), b_hi = min(b_lo + per, s.batch);
    long long mine = 0, before;
    int flags = 0, long_one = 0;
    SeqSpan span{0, 0, 0};   // by_warp: this lane's sequence
    for (int b = b_lo; b < b_hi; ++b) {
        int bit;
        span = seq_span(s, b, &bit);
        flags |= bit;
        const int nt = tiles(span.n);
        if (by_warp && nt > kFewTiles) {
            long_one = nt;
            continue;
        }
        for (int i = 0; i < nt; ++i) mine += (long long)units(span, i) * num_kv_heads;
    }
    if (by_warp) {
        // A sequence of many tiles is summed by all lanes.
        for (unsigned todo = __ballot_sync(0xffffffffu, long_one); todo; todo &= todo - 1) {
            const int src = __ffs(todo) - 1, nt = __shfl_sync(0xffffffffu, long_one, src);
            const SeqSpan q{__shfl_sync(0xffffffffu, span.row0, src), __shfl_sync(0xffffffffu, span.n, src),
                            __shfl_sync(0xffffffffu, span.ctx, src)};
            long long sum = 0;
            for (int i = lane; i < nt; i += 32) sum += units(q, i);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == src) mine = sum * num_kv_heads;
        }
        long long v = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += t;
        }
        *T = __shfl_sync(0xffffffffu, v, 31);
        before = v - mine;
        *bad = __any_sync(0xffffffffu, flags);
    } else {
        *bad = __syncthreads_or(flags);
        before = block_prefix(mine, tmp, T);
    }
    *n = *T >= (long long)workers * least ? workers : max(max((int)*T / least, min(min(items, workers), (int)*T)), 1);
    // T who / n from one division (of 32 bits where T allows): n^2 is small.
    const int k = *n;
    const long long each = *T < 0x80000000LL ? (int)*T / k : *T / k;
    const int rest = (int)(*T - each * k);
    *x0 = who < k ? who * each + who * rest / k : 0;
    *x1 = who < k ? (who + 1) * each + (who + 1) * rest / k : 0;
    const bool any = *x0 < *x1, snaps = *T <= (long long)k * mean;

    // The item that holds unit x < T, and its units in *item.
    auto locate = [&](long long x, int *item) {
        Start c{0, 0, 0, 0};
        int cu = 1;
        const bool here = before <= x && x < before + mine;
        if (here && !long_one) {
            long long rem = x - before;
            bool found = false;
            for (int b = b_lo; b < b_hi && !found; ++b) {
                int bit;
                const SeqSpan q = by_warp ? span : seq_span(s, b, &bit);
                const int nt = tiles(q.n);
                for (int i = 0; i < nt && !found; ++i) {
                    const int u = units(q, i);
                    if (rem < (long long)u * num_kv_heads) {
                        // rem < units of one tile x kv heads: fewer than 2^32 for any pool that fits in memory
                        c = {b, i, (int)((unsigned)rem / (unsigned)u), (int)((unsigned)rem % (unsigned)u)};
                        cu = u;
                        found = true;
                    }
                    rem -= (long long)u * num_kv_heads;
                }
            }
        }
        const unsigned in_long = by_warp ? __ballot_sync(0xffffffffu, here && long_one) : 0u;
        if (in_long) {   // 32 tiles at a time
            const int src = __ffs(in_long) - 1, nt = __shfl_sync(0xffffffffu, long_one, src);
            const SeqSpan q{__shfl_sync(0xffffffffu, span.row0, src), __shfl_sync(0xffffffffu, span.n, src),
                            __shfl_sync(0xffffffffu, span.ctx, src)};
            long long rem = __shfl_sync(0xffffffffu, x - before, src);
            for (int i0 = 0; i0 < nt; i0 += 32) {
                const int u = i0 + lane < nt ? units(q, i0 + lane) : 0;
                long long upto = (long long)u * num_kv_heads;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long t = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += t;
                }
                const unsigned past = __ballot_sync(0xffffffffu, rem < upto);
                if (past) {
                    const int at_lane = __ffs(past) - 1;
                    const long long start = __shfl_sync(0xffffffffu, upto - (long long)u * num_kv_heads, at_lane);
                    const unsigned left = (unsigned)(rem - start), ut = (unsigned)__shfl_sync(0xffffffffu, u, at_lane);
                    if (lane == src) {
                        c = {src, i0 + at_lane, (int)(left / ut), (int)(left % ut)};
                        cu = (int)ut;
                    }
                    break;
                }
                rem -= __shfl_sync(0xffffffffu, upto, 31);
            }
        }
        if (by_warp) {
            const int src = max(__ffs(__ballot_sync(0xffffffffu, here)) - 1, 0);
            c = {__shfl_sync(0xffffffffu, c.b, src), __shfl_sync(0xffffffffu, c.tile, src),
                 __shfl_sync(0xffffffffu, c.h, src), __shfl_sync(0xffffffffu, c.off, src)};
            cu = __shfl_sync(0xffffffffu, cu, src);
        } else {
            __syncthreads();
            if (here) {
                at[0] = c.b;
                at[1] = c.tile;
                at[2] = c.h;
                at[3] = c.off;
                at[4] = cu;
            }
            __syncthreads();
            c = {at[0], at[1], at[2], at[3]};
            cu = at[4];
        }
        *item = cu;
        return c;
    };
    Start c{0, 0, 0, 0};
    int item;
    if (!any) return c;
    if (snaps && *x1 < *T) {
        c = locate(*x1, &item);
        if (item <= snap) *x1 += 2 * c.off < item ? -c.off : item - c.off;
    }
    c = locate(*x0, &item);
    if (snaps && item <= snap) {
        const int to = 2 * c.off < item ? 0 : item;
        *x0 += to - c.off;
        c.off = to;
    }
    return c;
}

// Which CTA of n holds unit x of T.
__device__ __forceinline__ int cta_of_unit(long long x, long long T, int n) {
    return (int)(((x + 1) * n - 1) / T);
}

}  // namespace
}  // namespace hd
