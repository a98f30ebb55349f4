// Choice of the pages that a new token attends to.
//
// A block's score is the largest that its keys' bounds allow, summed over the
// heads that share it:
//     sum_g sum_d max(q_gd lo_d, q_gd hi_d) = Q+ . hi + Q- . lo,
// Q+ = sum_g max(q_g, 0), Q- = sum_g min(q_g, 0) -- one 512-term dot product
// per block instead of one per head.  The score kernel reads each block's
// bounds once (1 KiB); at long contexts that read bounds it, at half of
// DRAM's rate, as a warp has four blocks' bounds under way (64 rows of up to 1025
// blocks at 2 kv heads: 19 us; the pick 10 us, mostly latency).
//
// Which block is chosen must not hang on the order of a sum.  Scores are taken
// in binary32 first.  A score is sixteen terms a lane and five levels of a
// tree over the lanes, on Q+- that are sums of up to eight values: at most 28
// roundings on any term's way, so it is off by less than E = 32 2^-24 A, A the
// sum of the terms' magnitudes (kept beside the score, its own rounding inside
// the slack of 32 over 28).  With t the k-th largest score and E the row's
// largest bound, the exact k-th largest lies within E of t: blocks scored above
// t + 2E are chosen, below t - 2E not, and only those between -- mostly one or
// none more than are wanted -- are scored again with twice the digits:
// products split exactly by an fma, sums by the error-free addition of Knuth
// (The Art of Computer Programming, vol. 2, 4.2.2).  Ties go to the lower block.
#include <algorithm>

#include "paged_sched.cuh"

namespace hd {
namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kMaxBlocksPerWarp = 32;                                // of one score CTA; a multiple of kInFlight
constexpr int kInFlight = 4;                                         // blocks whose bounds a warp loads at once
constexpr int kPickThreads = 512;
constexpr float kErrUnits = 32.f * 5.9604645e-8f;

// a + b = s + e exactly.
__device__ __forceinline__ float two_sum(float a, float b, float &e) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
    return s;
}
// (h, l) += x, with x's rounding error left in l.
__device__ __forceinline__ void add_to(float &h, float &l, float x) {
    float e;
    h = two_sum(h, x, e);
    l = __fadd_rn(l, e);
}
// (h, l) += (qh + ql) b.
__device__ __forceinline__ void fma_to(float &h, float &l, float qh, float ql, float b) {
    const float p = __fmul_rn(qh, b);
    const float e = fmaf(qh, b, -p);
    add_to(h, l, p);
    l = __fadd_rn(l, fmaf(ql, b, e));
}
// Monotone integer keys.
__device__ __forceinline__ uint32_t key_of(float f) {
    const uint32_t u = __float_as_uint(f + 0.f);   // -0 ranks with +0
    return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float score_of(uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7FFFFFFFu : ~k); }
__device__ __forceinline__ uint64_t key_of(double d) {
    const uint64_t u = (uint64_t)__double_as_longlong(d + 0.0);
    return u >> 63 ? ~u : u | (1ull << 63);
}

// A lane's eight dims of Q+ and Q- in binary32, or in two parts each.
struct QuerySums {
    float ph[8], nh[8];
};
struct QuerySums2 {
    float ph[8], pl[8], nh[8], nl[8];
};
__device__ __forceinline__ float head_sign(const PagedSelectArgs &a, int h) {
    return a.k_scale && a.k_scale[h] < 0.f ? -1.f : 1.f;
}
__device__ __forceinline__ void sum_queries(const PagedSelectArgs &a, int r, int h, int lane, QuerySums &q) {
    const __nv_bfloat16 *src = a.q + ((size_t)r * a.num_q_heads + h * a.group) * kHeadDim + 8 * lane;
    const float sign = head_sign(a, h);
    uint4 raw[8];
#pragma unroll
    for (int g = 0; g < 8; ++g)
        raw[g] = g < a.group ? __ldg(reinterpret_cast<const uint4 *>(src + (size_t)g * kHeadDim)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int j = 0; j < 8; ++j) q.ph[j] = q.nh[j] = 0.f;
#pragma unroll
    for (int g = 0; g < 8; ++g) {
        float x[8];
        unpack_bf16x8(raw[g], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            q.ph[j] += fmaxf(x[j] * sign, 0.f);
            q.nh[j] += fminf(x[j] * sign, 0.f);
        }
    }
}
__device__ __forceinline__ void sum_queries(const PagedSelectArgs &a, int r, int h, int lane, QuerySums2 &q) {
    const __nv_bfloat16 *src = a.q + ((size_t)r * a.num_q_heads + h * a.group) * kHeadDim + 8 * lane;
    const float sign = head_sign(a, h);
#pragma unroll
    for (int j = 0; j < 8; ++j) q.ph[j] = q.pl[j] = q.nh[j] = q.nl[j] = 0.f;
    for (int g = 0; g < a.group; ++g) {
        float x[8];
        unpack_bf16x8(__ldg(reinterpret_cast<const uint4 *>(src + (size_t)g * kHeadDim)), x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            add_to(q.ph[j], q.pl[j], fmaxf(x[j] * sign, 0.f));
            add_to(q.nh[j], q.nl[j], fminf(x[j] * sign, 0.f));
        }
    }
}
__device__ __forceinline__ const uint4 *bounds_of(const PagedSelectArgs &a, int page, int h, int lane) {
    return reinterpret_cast<const uint4 *>(a.bounds + ((size_t)page * a.num_kv_heads + h) * 2 * kHeadDim) + lane;
}
// Whether block i of a token whose own block is `last` is chosen whatever its score.
__device__ __forceinline__ bool kept(const PagedSelectArgs &a, int i, int last) {
    return i < a.keep_first || i > last - a.keep_last;
}

// Grid: (row, kv head, chunk of 8 x per_warp blocks), the chunk fastest.  Scores go out as (score, A).
__global__ void __launch_bounds__(kScoreThreads, 4) page_score_kernel(const __grid_constant__ PagedSelectArgs a, int chunks,
                                                                     int per_warp) {
    wait_for_previous_kernel();
    let_next_kernel_start();
    const PagedSeqs &sq = a.seqs;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int chunk = blockIdx.x % chunks, rh = blockIdx.x / chunks;
    const int h = rh % a.num_kv_heads, r = rh / a.num_kv_heads;
    int bit, b;
    const SeqSpan q = span_of_row(sq, r, &bit, &b);
    if (q.n == 0) return;
    const int last = (q.ctx + r - q.row0) >> sq.page_shift;
    const int blk0 = (chunk * kScoreWarps + warp) * per_warp;
    if (blk0 > last) return;
    const int mine = blk0 + lane;
    int page = lane < per_warp && mine <= last ? sq.table[(size_t)b * sq.table_stride + mine] : 0;
    const bool valid = page >= 0 && page < sq.num_pages;
    if (!valid) {
        atomicOr(sq.err, HD_DEVERR_PAGE);
        page = 0;
    }
    const uint4 *lo_hi = bounds_of(a, 0, h, lane);
    const size_t per_page = (size_t)a.num_kv_heads * (2 * kHeadDim / 8);   // 16-byte words
    uint4 lo[kInFlight], hi[kInFlight];
    auto load = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            const uint4 *p = lo_hi + __shfl_sync(0xffffffffu, page, i0 + i) * per_page;
            const bool need = blk0 + i0 + i <= last;
            lo[i] = need ? __ldg(p) : make_uint4(0u, 0u, 0u, 0u);
            hi[i] = need ? __ldg(p + 32) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    load(0);   // under way while the queries are summed
    QuerySums s;
    sum_queries(a, r, h, lane, s);
    const unsigned good = __ballot_sync(0xffffffffu, valid);
    float *scores = reinterpret_cast<float *>(a.scores + (size_t)rh * a.score_stride);
#pragma unroll 1
    for (int i0 = 0; i0 < per_warp; i0 += kInFlight) {
        if (blk0 + i0 > last) break;
        if (i0) load(i0);
        float x[2 * kInFlight];   // score and A of each block
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            float l8[8], h8[8], v = 0.f, m = 0.f;
            unpack_bf16x8(lo[i], l8);
            unpack_bf16x8(hi[i], h8);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v = fmaf(s.ph[j], h8[j], v);
                m = fmaf(s.ph[j], fabsf(h8[j]), m);
                v = fmaf(s.nh[j], l8[j], v);
                m = fmaf(-s.nh[j], fabsf(l8[j]), m);
            }
            x[2 * i] = v;
            x[2 * i + 1] = m;
        }
        // Sum the eight values over the lanes, halving the values a lane is left with at each of the first three steps.
        static_assert(kInFlight == 4, "three halvings leave one value");
#pragma unroll
        for (int o = 16, n = 4; o >= 4; o >>= 1, n >>= 1) {
            const bool up = lane & o;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float send = up ? x[i] : x[i + n], keep = up ? x[i + n] : x[i];
                x[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
        }
        x[0] += __shfl_xor_sync(0xffffffffu, x[0], 2);
        x[0] += __shfl_xor_sync(0xffffffffu, x[0], 1);
        const int at = i0 + (lane >> 3), blk = blk0 + at, second = lane >> 2 & 1;   // lane's block, score or A
        if ((lane & 3) == 0 && at < per_warp && blk <= last) {
            float y = x[0];
            if (!(good >> at & 1)) y = second ? 0.f : -INFINITY;
            if (kept(a, blk, last)) y = second ? 0.f : INFINITY;
            scores[2 * blk + second] = y;
        }
    }
}

// The k-th largest of the keys that take(i) admits, most significant byte
// first: returns the prefix of its digits, `shift` the bits left of it, `want`
// how many of the keys with that prefix are among the k.  Ends as soon as a
// prefix's keys are all among them.
template <class K, class Take>
__device__ __forceinline__ K radix_select(const K *keys, int n, int k, Take take, int *hist, int *state, int *shift_out,
                                          int *want_out) {
    const int tid = threadIdx.x;
    K prefix = 0;
    int want = k, shift = 8 * (int)sizeof(K);
    while (shift > 0) {
        const bool first = shift == 8 * (int)sizeof(K);
        shift -= 8;
        for (int i = tid; i < 256; i += kPickThreads) hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kPickThreads)
            if (take(i) && (first || keys[i] >> (first ? 0 : shift + 8) == prefix)) atomicAdd(&hist[(int)(keys[i] >> shift) & 255], 1);
        __syncthreads();
        if (tid < 32) {   // the bucket where the running count from the top reaches `want`
            int c[8], sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += c[j] = hist[255 - (8 * tid + j)];
            int upto = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, upto, o);
                if (tid >= o) upto += t;
            }
            int above = upto - sum;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (above < want && want <= above + c[j]) {
                    state[0] = 255 - (8 * tid + j);
                    state[1] = want - above;
                    state[2] = c[j];
                }
                above += c[j];
            }
        }
        __syncthreads();
        prefix = (first ? (K)0 : (K)(prefix << 8)) | (K)state[0];
        want = state[1];
        const bool whole = want == state[2];
        __syncthreads();
        if (whole) break;
    }
    *shift_out = shift;
    *want_out = want;
    return prefix;
}

// One CTA per (row, kv head): the blocks of the num_selected largest scores, ascending, -1 behind them.
__global__ void __launch_bounds__(kPickThreads) page_pick_kernel(const __grid_constant__ PagedSelectArgs a, int max_blocks) {
    extern __shared__ uint64_t fine[];                             // exact keys of the blocks in doubt
    uint32_t *coarse = reinterpret_cast<uint32_t *>(fine + max_blocks);
    __shared__ int hist[256], state[3], edge_bits;
    __shared__ long long scan[33];
    const PagedSeqs &sq = a.seqs;
    const int tid = threadIdx.x, lane = tid & 31, rh = blockIdx.x, r = rh / a.num_kv_heads, h = rh % a.num_kv_heads;
    if (tid == 0) edge_bits = 0;
    wait_for_previous_kernel();
    let_next_kernel_start();
    int bit, b;
    const SeqSpan q = span_of_row(sq, r, &bit, &b);
    int32_t *out = a.selected + (size_t)rh * a.num_selected;
    if (q.n == 0) {
        // A row of a sequence that cannot be served: no block.  Rows behind the last sequence stay as they are.
        if (bit) {
            if (tid == 0) atomicOr(sq.err, bit);
            if (r >= q.row0)
                for (int i = tid; i < a.num_selected; i += kPickThreads) out[i] = -1;
        }
        return;
    }
    const int last = (q.ctx + r - q.row0) >> sq.page_shift, n = last + 1, k = min(a.num_selected, n);
    for (int i = k + tid; i < a.num_selected; i += kPickThreads) out[i] = -1;
    if (n == k) {
        for (int i = tid; i < n; i += kPickThreads) out[i] = i;
        return;
    }
    __syncthreads();
    float top = 0.f;
    for (int i = tid; i < n; i += kPickThreads) {
        const float2 s = a.scores[(size_t)rh * a.score_stride + i];
        coarse[i] = key_of(s.x);
        top = fmaxf(top, s.y);
    }
    atomicMax(&edge_bits, __float_as_int(top));   // not negative: ordered like its bits
    int shift, want;
    const uint32_t p32 = radix_select<uint32_t>(coarse, n, k, [](int) { return true; }, hist, state, &shift, &want);
    // Any score whose key has the prefix may be the k-th: take the doubt's band around all of them.
    const float err = 2.f * kErrUnits * __int_as_float(edge_bits);
    const float t_lo = score_of(p32 << shift), t_hi = score_of(p32 << shift | ((shift ? 1u << shift : 1u) - 1u));
    // Sure: above the band, or (radix ended early) every key with the prefix when nothing below comes near.
    auto above = [&](int i) { return score_of(coarse[i]) > t_hi + err; };
    auto below = [&](int i) { return score_of(coarse[i]) < t_lo - err; };
    int sure = 0, open = 0;
    for (int i = tid; i < n; i += kPickThreads) {
        const bool up = above(i);
        sure += up;
        open += !up && !below(i);
    }
    long long counts;
    block_prefix((long long)sure << 32 | open, scan, &counts);
    sure = (int)(counts >> 32);
    open = (int)(counts & 0xFFFFFFFF);
    uint64_t prefix = 0;
    int fshift = 64, fwant = open;   // all of the open ones, unless there are more than are wanted
    if (open > k - sure) {
        QuerySums2 s;
        sum_queries(a, r, h, lane, s);
        const int32_t *row = sq.table + (size_t)b * sq.table_stride;
        __syncthreads();   // hist and state are free
        for (int i0 = 32 * (tid >> 5); i0 < n; i0 += kPickThreads) {
            const int i = i0 + lane;
            unsigned todo = __ballot_sync(0xffffffffu, i < n && !above(i) && !below(i));
            while (todo) {
                const int j = i0 + __ffs(todo) - 1;
                todo &= todo - 1;
                uint64_t key = ~0ull;
                const int page = row[j];
                if (!kept(a, j, last)) {
                    key = 0;
                    if (page >= 0 && page < sq.num_pages) {
                        const uint4 *p = bounds_of(a, page, h, lane);
                        float l8[8], h8[8], sh = 0.f, sl = 0.f;
                        unpack_bf16x8(__ldg(p), l8);
                        unpack_bf16x8(__ldg(p + 32), h8);
#pragma unroll
                        for (int d = 0; d < 8; ++d) {
                            fma_to(sh, sl, s.ph[d], s.pl[d], h8[d]);
                            fma_to(sh, sl, s.nh[d], s.nl[d], l8[d]);
                        }
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1) {
                            const float xh = __shfl_xor_sync(0xffffffffu, sh, o), xl = __shfl_xor_sync(0xffffffffu, sl, o);
                            float e;
                            sh = two_sum(sh, xh, e);
                            sl = __fadd_rn(__fadd_rn(sl, xl), e);
                        }
                        key = key_of((double)sh + (double)sl);
                    }
                }
                if (lane == 0) fine[j] = key;
            }
        }
        __syncthreads();
        prefix = radix_select<uint64_t>(fine, n, k - sure, [&](int i) { return !above(i) && !below(i); }, hist, state, &fshift,
                                        &fwant);
    }
    // Each thread takes a run of blocks; its place in the list is what the runs before it hold.
    const int per = (n + kPickThreads - 1) / kPickThreads, lo = min(n, tid * per), hi = min(n, lo + per);
    auto rank = [&](int i) {   // 2: chosen, 1: chosen while some are wanted, 0: not
        if (above(i)) return 2;
        if (below(i)) return 0;
        if (fshift == 64) return 2;
        const uint64_t t = fine[i] >> fshift;
        return t > prefix ? 2 : t == prefix ? 1 : 0;
    };
    int chosen = 0, equal = 0;
    for (int i = lo; i < hi; ++i) {
        const int x = rank(i);
        chosen += x == 2;
        equal += x == 1;
    }
    long long total;
    __syncthreads();   // the first count's readers of scan are through
    const long long before = block_prefix((long long)chosen << 32 | equal, scan, &total);
    chosen = (int)(before >> 32);
    equal = (int)(before & 0xFFFFFFFF);
    for (int i = lo; i < hi; ++i) {
        const int x = rank(i);
        if (x == 2 || (x == 1 && equal < fwant)) out[chosen + min(equal, fwant)] = i;
        chosen += x == 2;
        equal += x == 1;
    }
}

}  // namespace

cudaError_t launch_paged_select(const PagedSelectArgs &a, int max_blocks, int num_sms, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (!done_on_device(done, &dev)) {
        const cudaError_t e = cudaFuncSetAttribute(page_pick_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kMaxSelectBlocks * 12);
        if (e != cudaSuccess) return e;
        mark_done_on_device(done, dev);
    }
    // A warp's blocks: enough warps to fill the SMs one and a half times over (32 each), then longer runs, which share
    // a look-up of the position and the sums of the queries (4 rows of 2049 blocks at 2 kv heads: 4 blocks 8.9 us,
    // 16 blocks 10.9 us; 64 rows of up to 1025: 20 blocks).
    const long long rh = (long long)a.seqs.num_tokens * a.num_kv_heads;
    const long long even = (rh * max_blocks + 48LL * num_sms - 1) / (48LL * num_sms);
    const int per_warp = (int)std::min<long long>(kMaxBlocksPerWarp, (even + kInFlight - 1) / kInFlight * kInFlight);
    const int chunks = (max_blocks + kScoreWarps * per_warp - 1) / (kScoreWarps * per_warp);
    if (rh * chunks > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
    const cudaError_t e = launch_overlapping(page_score_kernel, dim3((unsigned)(rh * chunks)), kScoreThreads, 0, 1, s, a, chunks, per_warp);
    if (e != cudaSuccess) return e;
    return launch_overlapping(page_pick_kernel, dim3((unsigned)rh), kPickThreads, (size_t)max_blocks * 12, 1, s, a, max_blocks);
}

}  // namespace hd
