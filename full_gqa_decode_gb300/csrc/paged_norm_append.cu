// Append to a paged cache with the heads' norms and a given table of angles:
// norm, rotation, store and the pages' key bounds in one pass.
//
//     y = x rsqrt(mean(x^2) + eps) (offset + weight),   z = rotation of y
//
// Bytes: q, k, v and a row's angles once in; q and the entries once out.  A warp
// takes a 256-dim row, eight dims a lane so that a pair's two dims sit in one
// lane: dims 4l .. 4l+3 and their partners half a rotation on (halves), or eight
// neighbours.  The mean is one warp-wide sum of eight squares a lane.  Query
// rows go four heads to a warp, which share the row's angles and hide one
// another's sums; keys and values go by runs -- the new tokens of one page and
// kv head, one CTA, which owns the page's bounds -- two rows a warp at a time.
// Bound by the latency of its chains of loads (offsets, context, angles): four
// CTAs an SM at 64 registers, some 50 bytes a thread spilled, beat both fewer and
// larger warps.  Measured: a packed prompt of 16384 tokens 38.2 us (5.7 TB/s, 86 % of a
// copy's rate; at 80 registers 42.7, eight heads a warp 39.5, five CTAs 44), 9026 tokens
// at 16 heads over E4M3 pages 36.8 us (5.0 TB/s), one token of 64 sequences 2.9 us from
// a graph.
#include <climits>

#include "paged_entry.cuh"

namespace hd {
namespace {

constexpr int kHeads = 4;   // query heads of a row that one warp takes
constexpr int kRows = 2;    // rows of a run that one warp has under way

// A lane's eight dims of a row, and the row's angles that go with them.
template <bool NEIGHBOURS>
__device__ __forceinline__ LaneDims norm_lane_dims(int lane, int rot) {
    if (!NEIGHBOURS) return lane_dims(lane, rot);
    return {8 * lane, 8 * lane + 4, 8 * lane < rot ? 4 * lane : -1};
}
template <bool NEIGHBOURS>
__device__ __forceinline__ uint4 load_dims(const __nv_bfloat16 *row, const LaneDims &ld) {
    if (NEIGHBOURS) return *reinterpret_cast<const uint4 *>(row + ld.d0);
    const uint2 x = *reinterpret_cast<const uint2 *>(row + ld.d0), y = *reinterpret_cast<const uint2 *>(row + ld.d1);
    return make_uint4(x.x, x.y, y.x, y.y);
}
template <bool NEIGHBOURS>
__device__ __forceinline__ void store_dims(__nv_bfloat16 *row, const LaneDims &ld, const uint4 &w) {
    if (NEIGHBOURS) {
        *reinterpret_cast<uint4 *>(row + ld.d0) = w;
    } else {
        *reinterpret_cast<uint2 *>(row + ld.d0) = make_uint2(w.x, w.y);
        *reinterpret_cast<uint2 *>(row + ld.d1) = make_uint2(w.z, w.w);
    }
}

// offset + weight of a lane's dims (1 without weights).
__device__ __forceinline__ void load_weights(const void *w, bool f32, float offset, const LaneDims &ld, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 1.f;
    if (!w) return;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int d = half ? ld.d1 : ld.d0;
        float u[4];
        if (f32) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(w) + d));
            u[0] = v.x; u[1] = v.y; u[2] = v.z; u[3] = v.w;
        } else {
            unpack4(__ldg(reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(w) + d)), u);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) x[4 * half + j] = offset + u[j];
    }
}
__device__ __forceinline__ const void *weights_of(const void *w, const PagedNormArgs &a, int head) {
    if (!w || !a.per_head) return w;
    return static_cast<const uint8_t *>(w) + (size_t)head * kHeadDim * (a.f32_weights ? 4 : 2);
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// A lane's dims of the normed and rotated row (every lane of the warp calls it).
template <bool NEIGHBOURS>
__device__ __forceinline__ void norm_rotate(const PagedNormArgs &a, const uint4 &raw, const float (&w)[8], const float (&c)[4],
                                            const float (&s)[4], bool turned, float (&y)[8]) {
    unpack_bf16x8(raw, y);
    if (a.norm) {
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sq = fmaf(y[i], y[i], sq);
        // The mean in two steps of 2^-4: the sum of a whole head of values of 2^60 alone is infinite.
        const float r = rsqrtf(fmaf(warp_sum(sq * (1.f / 16)), 16.f / kHeadDim, a.eps));
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = y[i] * r * w[i];
    }
    if (!turned) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int p = NEIGHBOURS ? 2 * j : j, q = NEIGHBOURS ? 2 * j + 1 : 4 + j;
        const float x1 = y[p], x2 = y[q];
        y[p] = x1 * c[j] - x2 * s[j];
        y[q] = x2 * c[j] + x1 * s[j];
    }
}
__device__ __forceinline__ uint4 to_bf16(const float (&y)[8]) {
    return make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
}

// A call, as it is hardly ever wanted.
__device__ __noinline__ float quotient(float x, float y) { return __fdiv_rn(x, y); }

// The table row of new token r, at position p: -1 when a given position is not in the table.
__device__ __forceinline__ int angle_row(const PagedNormArgs &a, int r, int p) {
    if (!a.positions) return p;
    const int t = a.positions[r];
    return t >= 0 && t < a.table_rows ? t : -1;
}

template <bool NEIGHBOURS>
__global__ void __launch_bounds__(kEntryThreads, 4) paged_norm_append_kernel(const __grid_constant__ PagedNormArgs a, int runs) {
    const PagedAppendArgs &e = a.entry;
    const PagedSeqs &sq = e.seqs;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int half = e.rotary_dim >> 1, ps = 1 << sq.page_shift;
    const LaneDims ld = norm_lane_dims<NEIGHBOURS>(lane, e.rotary_dim);
    __shared__ long long scan[33];
    __shared__ int found[2];
    __shared__ float edge[2][kEntryWarps][kHeadDim];
    wait_for_previous_kernel();
    let_next_kernel_start();

    if ((int)blockIdx.x >= runs * e.num_kv_heads) {
        // ---- queries: a warp takes up to kHeads heads of a row ----
        const int parts = (e.num_q_heads + kHeads - 1) / kHeads;
        const long long vec = (long long)(blockIdx.x - runs * e.num_kv_heads) * kEntryWarps + warp;
        const int r = (int)(vec / parts), h0 = (int)(vec % parts) * kHeads;
        if (r >= sq.num_tokens) return;
        const __nv_bfloat16 *src = e.q + (size_t)r * e.q_stride + h0 * kHeadDim;
        __nv_bfloat16 *dst = e.q_rot + ((size_t)r * e.num_q_heads + h0) * kHeadDim;
        const int heads = min(kHeads, e.num_q_heads - h0);
        uint4 x[kHeads];   // under way while the row's position is looked up
#pragma unroll
        for (int i = 0; i < kHeads; ++i) x[i] = i < heads ? load_dims<NEIGHBOURS>(src + i * kHeadDim, ld) : make_uint4(0u, 0u, 0u, 0u);
        int bit;
        const SeqSpan q = span_of_row(sq, r, &bit);
        if (q.n == 0) return;
        const int at = angle_row(a, r, q.ctx + r - q.row0);
        if (at < 0) {
            if (lane == 0) atomicOr(sq.err, HD_DEVERR_CONTEXT_PLAN);
            return;
        }
        float c[4] = {}, s[4] = {}, w[8];
        if (ld.i >= 0) load_angles(e.rope + (size_t)at * half, ld.i, c, s);
        load_weights(weights_of(a.q_weight, a, h0), a.f32_weights, a.offset, ld, w);
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            if (i >= heads) break;
            if (i && a.per_head) load_weights(weights_of(a.q_weight, a, h0 + i), a.f32_weights, a.offset, ld, w);
            float y[8];
            norm_rotate<NEIGHBOURS>(a, x[i], w, c, s, ld.i >= 0, y);
            store_dims<NEIGHBOURS>(dst + i * kHeadDim, ld, to_bf16(y));
        }
        return;
    }

    // ---- keys and values of one run ----
    const int run = blockIdx.x / e.num_kv_heads, h = blockIdx.x % e.num_kv_heads;
    int b, block;
    SeqSpan q;
    if (!find_run(sq, run, h == 0, scan, found, &b, &block, &q)) return;
    const int page = sq.table[(size_t)b * sq.table_stride + block];
    if (page < 0 || page >= sq.num_pages) {
        if (tid == 0) atomicOr(sq.err, HD_DEVERR_PAGE);
        return;
    }
    const int p0 = max(q.ctx, block << sq.page_shift), p1 = min(q.ctx + q.n, (block + 1) << sq.page_shift);
    const bool fp8 = e.kv_type == KV_FP8;
    const Recip vr = recip_of(fp8 ? e.v_scale[h] : 1.f);
    const float k_inv = fp8 ? 1.f / e.k_scale[h] : 1.f;
    const bool no_inv = fp8 && recip_of(e.k_scale[h]).odd;
    float w[8];
    load_weights(weights_of(a.k_weight, a, h), a.f32_weights, a.offset, ld, w);
    uint32_t lo[4], hi[4];   // of the keys' dims: bf16 pairs, or f16 pairs, which hold every E4M3 value
    const uint32_t inf = fp8 ? 0x7C007C00u : 0x7F807F80u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        lo[j] = inf;
        hi[j] = inf | 0x80008000u;
    }
    for (int p = p0 + warp; p < p1; p += kRows * kEntryWarps) {
        uint4 x[kRows], v[kRows];
        int at[kRows];
        float c[kRows][4] = {}, s[kRows][4] = {};
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int pos = min(p + i * kEntryWarps, p1 - 1), r = q.row0 + pos - q.ctx;   // the last row may come twice
            x[i] = load_dims<NEIGHBOURS>(e.k + (size_t)r * e.k_stride + h * kHeadDim, ld);
            v[i] = *reinterpret_cast<const uint4 *>(e.v + (size_t)r * e.v_stride + h * kHeadDim + 8 * lane);
            at[i] = angle_row(a, r, pos);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (ld.i >= 0 && at[i] >= 0) load_angles(e.rope + (size_t)at[i] * half, ld.i, c[i], s[i]);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int pos = p + i * kEntryWarps;
            if (pos >= p1) break;
            if (at[i] < 0) {
                if (lane == 0) atomicOr(sq.err, HD_DEVERR_CONTEXT_PLAN);
                continue;
            }
            float y[8];
            norm_rotate<NEIGHBOURS>(a, x[i], w, c[i], s[i], ld.i >= 0, y);
            const size_t o = (size_t)page * e.page_stride + ((size_t)h * ps + (pos & (ps - 1))) * kHeadDim;
            if (fp8) {
                // Codes of y times the scale's reciprocal: two more roundings to 2^-24 before the one to E4M3.  Of their
                // quotient where the reciprocal is no normal number: infinite, it would make a NaN of a zero.
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = no_inv ? quotient(y[j], e.k_scale[h]) : y[j] * k_inv;
                const uint32_t cx = e4m3x4(y[0], y[1], y[2], y[3]), cy = e4m3x4(y[4], y[5], y[6], y[7]);
                uint8_t *kd = static_cast<uint8_t *>(e.cache_k) + o;
                if (NEIGHBOURS) {
                    *reinterpret_cast<uint2 *>(kd + ld.d0) = make_uint2(cx, cy);
                } else {
                    *reinterpret_cast<uint32_t *>(kd + ld.d0) = cx;
                    *reinterpret_cast<uint32_t *>(kd + ld.d1) = cy;
                }
                float f[8];
                unpack_bf16x8(v[i], f);
                const float v0[4] = {f[0], f[1], f[2], f[3]}, v1[4] = {f[4], f[5], f[6], f[7]};
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(e.cache_v) + o + 8 * lane) =
                    make_uint2(e4m3_plain(v0, vr), e4m3_plain(v1, vr));
                widen2<false>(lo[0], hi[0], e4m3x2_to_f16x2(cx & 0xFFFFu));
                widen2<false>(lo[1], hi[1], e4m3x2_to_f16x2(cx >> 16));
                widen2<false>(lo[2], hi[2], e4m3x2_to_f16x2(cy & 0xFFFFu));
                widen2<false>(lo[3], hi[3], e4m3x2_to_f16x2(cy >> 16));
            } else {
                const uint4 k = to_bf16(y);
                store_dims<NEIGHBOURS>(static_cast<__nv_bfloat16 *>(e.cache_k) + o, ld, k);
                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(e.cache_v) + o + 8 * lane) = v[i];
                widen2<true>(lo[0], hi[0], k.x);
                widen2<true>(lo[1], hi[1], k.y);
                widen2<true>(lo[2], hi[2], k.z);
                widen2<true>(lo[3], hi[3], k.w);
            }
        }
    }
    if (!e.bounds) return;
    bool fresh = (p0 & (ps - 1)) == 0;
    if (a.positions) {   // rows that were not stored leave the bounds as they are: a thread looks at each
        static_assert(kEntryThreads >= 1 << kMaxPageShift, "a run has at most as many rows as a CTA threads");
        const int pos = p0 + tid, r0 = q.row0 - q.ctx;
        if (!__syncthreads_or(pos < p1 && angle_row(a, r0 + pos, pos) >= 0)) return;
        fresh = fresh && angle_row(a, r0 + p0, p0) >= 0;
    }
    store_bounds(e, page, h, fp8, fresh, ld, lo, hi, edge);
}

}  // namespace

cudaError_t launch_paged_norm_append(const PagedNormArgs &a, cudaStream_t s) {
    const PagedAppendArgs &e = a.entry;
    const long long runs = max_runs(e.seqs), parts = (e.num_q_heads + kHeads - 1) / kHeads;
    const long long qctas = e.q ? ((long long)e.seqs.num_tokens * parts + kEntryWarps - 1) / kEntryWarps : 0;
    const long long grid = runs * e.num_kv_heads + qctas;
    if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
    return launch_overlapping(a.neighbours ? paged_norm_append_kernel<true> : paged_norm_append_kernel<false>,
                              dim3((unsigned)grid), kEntryThreads, 0, 1, s, a, (int)runs);
}

}  // namespace hd
