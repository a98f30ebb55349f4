// Choice of the pages that a new token attends to.
//
// A block's score is the largest that its keys' bounds allow, summed over the
// heads that share it:
//     sum_g sum_d max(q_gd lo_d, q_gd hi_d) = Q+ . hi + Q- . lo,
// Q+ = sum_g max(q_g, 0), Q- = sum_g min(q_g, 0) -- one 512-term dot product
// per block instead of one per head.  The kernel reads each block's bounds once
// (1 KiB); at long contexts that read bounds it.
//
// Which block is chosen must not hang on the order of a sum, so scores carry
// twice binary32's digits: products split exactly by an fma, sums by the
// error-free addition of Knuth (The Art of Computer Programming, vol. 2,
// 4.2.2), which is far cheaper here than binary64 (a sixtieth of the binary32
// rate).  The two parts meet in a binary64 value whose bits, made monotone, are
// the ranking key; ties go to the lower block.  The k-th key is found by radix
// passes over the keys in shared memory, most significant byte first, ending as
// soon as a byte's bucket is taken whole.
#include "paged_sched.cuh"

namespace hd {
namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kBlocksPerWarp = 8;                                    // of one score CTA
constexpr int kBlocksPerCta = kScoreWarps * kBlocksPerWarp;
constexpr int kPickThreads = 512;

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

__device__ __forceinline__ uint64_t ranking_key(double d) {
    const uint64_t u = (uint64_t)__double_as_longlong(d + 0.0);   // -0 ranks with +0
    return u >> 63 ? ~u : u | (1ull << 63);
}

// Grid: (row, kv head, chunk of kBlocksPerCta blocks), the chunk fastest.
__global__ void __launch_bounds__(kScoreThreads) page_score_kernel(const __grid_constant__ PagedSelectArgs a, int chunks) {
    const PagedSeqs &sq = a.seqs;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int chunk = blockIdx.x % chunks, rh = blockIdx.x / chunks;
    const int h = rh % a.num_kv_heads, r = rh / a.num_kv_heads;
    int bit, b;
    const SeqSpan q = span_of_row(sq, r, &bit, &b);
    if (q.n == 0) return;
    const int last = (q.ctx + r - q.row0) >> sq.page_shift;
    const int blk0 = chunk * kBlocksPerCta + warp * kBlocksPerWarp;
    if (blk0 > last) return;
    // This lane's eight dims of Q+ and Q-, each a sum in two parts.
    float ph[8], pl[8], nh[8], nl[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) ph[j] = pl[j] = nh[j] = nl[j] = 0.f;
    const bool turn = a.k_scale && a.k_scale[h] < 0.f;
    const __nv_bfloat16 *src = a.q + ((size_t)r * a.num_q_heads + h * a.group) * kHeadDim + 8 * lane;
    for (int g = 0; g < a.group; ++g) {
        float x[8];
        unpack_bf16x8(__ldg(reinterpret_cast<const uint4 *>(src + (size_t)g * kHeadDim)), x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = turn ? -x[j] : x[j];
            add_to(ph[j], pl[j], fmaxf(v, 0.f));
            add_to(nh[j], nl[j], fminf(v, 0.f));
        }
    }
    const int32_t *row = sq.table + (size_t)b * sq.table_stride;
    const int mine = blk0 + (lane & (kBlocksPerWarp - 1));
    int page = mine <= last ? row[mine] : 0;
    const bool valid = page >= 0 && page < sq.num_pages;
    if (!valid) {
        atomicOr(sq.err, HD_DEVERR_PAGE);
        page = 0;
    }
    const unsigned good = __ballot_sync(0xffffffffu, valid);
    uint64_t out = 0;
#pragma unroll
    for (int i0 = 0; i0 < kBlocksPerWarp; i0 += 4) {
        uint4 lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int pg = __shfl_sync(0xffffffffu, page, i0 + i);
            const uint4 *p = reinterpret_cast<const uint4 *>(a.bounds + ((size_t)pg * a.num_kv_heads + h) * 2 * kHeadDim) + lane;
            const bool need = blk0 + i0 + i <= last;
            lo[i] = need ? __ldg(p) : make_uint4(0u, 0u, 0u, 0u);
            hi[i] = need ? __ldg(p + 32) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float l8[8], h8[8], sh = 0.f, sl = 0.f;
            unpack_bf16x8(lo[i], l8);
            unpack_bf16x8(hi[i], h8);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                fma_to(sh, sl, ph[j], pl[j], h8[j]);
                fma_to(sh, sl, nh[j], nl[j], l8[j]);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float xh = __shfl_xor_sync(0xffffffffu, sh, o), xl = __shfl_xor_sync(0xffffffffu, sl, o);
                float e;
                sh = two_sum(sh, xh, e);
                sl = __fadd_rn(__fadd_rn(sl, xl), e);
            }
            if (lane == i0 + i) out = ranking_key((double)sh + (double)sl);
        }
    }
    if (lane < kBlocksPerWarp && mine <= last) {
        if (!(good >> lane & 1)) out = 0;
        if (mine < a.keep_first || mine > last - a.keep_last) out = ~0ull;   // always chosen
        a.scores[(size_t)rh * a.score_stride + mine] = out;
    }
}

// One CTA per (row, kv head): the blocks of the num_selected largest keys, ascending, -1 behind them.
__global__ void __launch_bounds__(kPickThreads) page_pick_kernel(const __grid_constant__ PagedSelectArgs a) {
    extern __shared__ uint64_t keys[];
    __shared__ int hist[256];
    __shared__ long long scan[33];
    __shared__ int state[2];   // bucket and what is still wanted from it
    const PagedSeqs &sq = a.seqs;
    const int tid = threadIdx.x, rh = blockIdx.x, r = rh / a.num_kv_heads;
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
    const int n = ((q.ctx + r - q.row0) >> sq.page_shift) + 1, k = min(a.num_selected, n);
    for (int i = k + tid; i < a.num_selected; i += kPickThreads) out[i] = -1;
    if (n == k) {
        for (int i = tid; i < n; i += kPickThreads) out[i] = i;
        return;
    }
    for (int i = tid; i < n; i += kPickThreads) keys[i] = a.scores[(size_t)rh * a.score_stride + i];
    uint64_t prefix = 0;
    int want = k, shift = 64;   // keys whose top (64 - shift) bits exceed prefix are chosen; `want` more from those equal
    while (shift > 0) {
        shift -= 8;
        for (int i = tid; i < 256; i += kPickThreads) hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kPickThreads)
            if (shift == 56 || keys[i] >> (shift + 8) == prefix) atomicAdd(&hist[keys[i] >> shift & 255], 1);
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
                }
                above += c[j];
            }
        }
        __syncthreads();
        prefix = prefix << 8 | (uint64_t)state[0];
        want = state[1];
        if (want == hist[state[0]]) break;   // the bucket is taken whole
        __syncthreads();
    }
    // Each thread takes a run of blocks; its place in the list is what the runs before it hold.
    const int per = (n + kPickThreads - 1) / kPickThreads, lo = min(n, tid * per), hi = min(n, lo + per);
    int above = 0, equal = 0;
    for (int i = lo; i < hi; ++i) {
        const uint64_t t = keys[i] >> shift;
        above += t > prefix;
        equal += t == prefix;
    }
    long long total;
    const long long before = block_prefix((long long)above << 32 | equal, scan, &total);
    above = (int)(before >> 32);
    equal = (int)(before & 0xFFFFFFFF);
    for (int i = lo; i < hi; ++i) {
        const uint64_t t = keys[i] >> shift;
        if (t > prefix || (t == prefix && equal < want)) out[above + min(equal, want)] = i;
        above += t > prefix;
        equal += t == prefix;
    }
}

}  // namespace

cudaError_t launch_paged_select(const PagedSelectArgs &a, int max_blocks, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (!done_on_device(done, &dev)) {
        const cudaError_t e = cudaFuncSetAttribute(page_pick_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kMaxSelectBlocks * 8);
        if (e != cudaSuccess) return e;
        mark_done_on_device(done, dev);
    }
    const int chunks = (max_blocks + kBlocksPerCta - 1) / kBlocksPerCta;
    const long long rh = (long long)a.seqs.num_tokens * a.num_kv_heads;
    if (rh * chunks > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
    page_score_kernel<<<(unsigned)(rh * chunks), kScoreThreads, 0, s>>>(a, chunks);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    page_pick_kernel<<<(unsigned)rh, kPickThreads, (size_t)max_blocks * 8, s>>>(a);
    return cudaGetLastError();
}

}  // namespace hd
