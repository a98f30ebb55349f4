// Reading a paged cache's entries back as rows in bf16.
//
// Bytes: the entries once in, the rows once out; nothing else bounds it.  A warp
// takes two neighbouring rows, which mostly lie in one sequence and page, and K
// and V of one head of them at a time: four independent loads a lane before the
// first store, at six CTAs an SM.  Measured: four sequences of up to 32768 over
// E4M3 pages 60.6 us (6.0 TB/s, 90 % of a copy's rate; four rows a warp 67.5, one
// 64.6), over bf16 pages 75 us (6.5 TB/s).
#include <climits>

#include "paged_sched.cuh"

namespace hd {
namespace {

constexpr int kReadThreads = 256, kReadWarps = kReadThreads / 32;
constexpr int kReadRows = 2;

// Eight codes of a lane as bf16: their values times the scale, rounded once.  The product of 4 and 24 bits is first rounded to
// odd in binary32 (towards zero, the last bit set where that was not exact), which the rounding to bf16 then takes as exact.
__device__ __forceinline__ uint4 scaled_codes(const uint2 &codes, float scale) {
    float f[8];
    unpack_e4m3x8(codes, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = __fmul_rz(f[i], scale);
        f[i] = __fmaf_rn(f[i], scale, -t) != 0.f ? __uint_as_float(__float_as_uint(t) | 1u) : t;
    }
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

template <int KV>
__global__ void __launch_bounds__(kReadThreads, 6) paged_read_kernel(const __grid_constant__ PagedReadArgs a) {
    constexpr bool kFp8 = KV == KV_FP8;
    const PagedSeqs &sq = a.seqs;
    const int lane = threadIdx.x & 31, ps = 1 << sq.page_shift;
    wait_for_previous_kernel();
    let_next_kernel_start();
    const long long first = ((long long)blockIdx.x * kReadWarps + (threadIdx.x >> 5)) * kReadRows;
    if (first >= sq.num_tokens) return;
    // Where each row's entry lies: -1 zeros (no such page), -2 NaN (a sequence that cannot be served), -3 no sequence's row.
    int64_t at[kReadRows];
    SeqSpan q{0, 0, 0};
    int seq = 0;
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
        const int r = (int)first + i;
        at[i] = -3;
        if (r >= sq.num_tokens) continue;
        int bit = 0;
        if (q.n == 0 || r < q.row0 || r >= q.row0 + q.n) q = span_of_row(sq, r, &bit, &seq);
        if (bit && lane == 0) atomicOr(sq.err, bit);
        if (q.n == 0) {
            if (bit && q.row0 <= r) at[i] = -2;
            continue;
        }
        const int p = q.ctx + r - q.row0, page = sq.table[(size_t)seq * sq.table_stride + (p >> sq.page_shift)];
        at[i] = -1;
        if (page >= 0 && page < sq.num_pages) at[i] = page * a.page_stride + (int64_t)(p & (ps - 1)) * kHeadDim + 8 * lane;
        else if (lane == 0) atomicOr(sq.err, HD_DEVERR_PAGE);
    }
    for (int h = 0; h < a.num_kv_heads; ++h) {
        uint4 x[kReadRows][2];
#pragma unroll
        for (int i = 0; i < kReadRows; ++i)
#pragma unroll
            for (int kind = 0; kind < 2; ++kind) {
                const uint32_t fill = at[i] == -2 ? 0x7FFF7FFFu : 0u;
                x[i][kind] = make_uint4(fill, fill, fill, fill);
                const void *cache = kind ? a.cache_v : a.cache_k;
                if (at[i] < 0 || !(kind ? a.v : a.k)) continue;
                const int64_t o = at[i] + (int64_t)h * ps * kHeadDim;
                if (kFp8) {
                    const uint2 c = __ldcs(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(cache) + o));
                    x[i][kind].x = c.x;
                    x[i][kind].y = c.y;
                } else {
                    x[i][kind] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(cache) + o));
                }
            }
        const float ks = kFp8 ? a.k_scale[h] : 1.f, vs = kFp8 ? a.v_scale[h] : 1.f;
#pragma unroll
        for (int i = 0; i < kReadRows; ++i) {
            if (at[i] == -3) continue;
            const int64_t r = first + i;
#pragma unroll
            for (int kind = 0; kind < 2; ++kind) {
                __nv_bfloat16 *dst = kind ? a.v : a.k;
                if (!dst) continue;
                uint4 w = x[i][kind];
                if (kFp8 && at[i] >= 0) w = scaled_codes(make_uint2(w.x, w.y), kind ? vs : ks);
                *reinterpret_cast<uint4 *>(dst + r * (kind ? a.v_stride : a.k_stride) + h * kHeadDim + 8 * lane) = w;
            }
        }
    }
}

}  // namespace

cudaError_t launch_paged_read(const PagedReadArgs &a, cudaStream_t s) {
    const long long warps = ((long long)a.seqs.num_tokens + kReadRows - 1) / kReadRows;
    const unsigned grid = (unsigned)((warps + kReadWarps - 1) / kReadWarps);
    return launch_overlapping(a.kv_type == KV_FP8 ? paged_read_kernel<KV_FP8> : paged_read_kernel<KV_BF16>, dim3(grid), kReadThreads,
                              0, 1, s, a);
}

}  // namespace hd
