// Append to a paged cache: rotation of the new queries and keys, the store of
// keys and values into their pages, and the pages' elementwise key bounds.
//
// Bytes: q, k, v once in; q and the entries once out.  One warp takes one
// 256-dim row, eight dims a lane arranged so that both halves of a rotary pair
// sit in one lane (lane l < rot/8: dims 4l .. 4l+3 and their partners at
// + rot/2; the other lanes: the dims past the rotation), so a row is read and
// written once, in 8-byte pieces.  Keys go by runs -- the new tokens of one
// page and kv head, one CTA -- because a run owns its page's bounds: the
// minimum and maximum over its keys stay in registers, merge across the warps
// in shared memory, and meet the bounds that the page had (a run that starts
// at slot 0 starts them anew).  No atomics, so results never depend on order.
//
// The written key is the exact rotation, rounded to binary64 and then to the
// entry's type.  GB300 runs binary64 at a sixtieth of the binary32 rate, so
// every value is first enclosed in binary32: an interval that holds the exact
// value, from the error bounds of its two or three operations.  Rounding is
// monotone, so when both ends round to the same entry that is the entry; only
// the others are evaluated in binary64 (about one bf16 value in four thousand,
// one E4M3 value in a hundred thousand).  The call is bound by the instructions
// of this, not by its bytes: testing each value's distance from the rounding's
// midpoint instead took twice as many (9026 tokens at 16 heads, E4M3: 71 us,
// so 37 us).
#include "paged_entry.cuh"

namespace hd {
namespace {

constexpr int kThreads = kEntryThreads, kWarps = kEntryWarps;
constexpr int kQueryHeads = 4;   // heads of a row that one warp rotates (9026 tokens at 16 heads: 2 44 us, 4 37 us)

// The binary64 paths are calls, see e4m3_rotated_f64.
__device__ __noinline__ uint32_t rotated_f64(float a, float c, float b, float s) {
    return __float_as_uint(f64_to_bf16_value(__dsub_rn(__dmul_rn((double)a, (double)c), __dmul_rn((double)b, (double)s)))) >> 16;
}

// bf16 of a c - b s, rounded once, for two pairs (a, b).  q = RN(b s) and y = fma(a, c, -q) are off by 2^-24 (|y| + |q|)
// and, where they are subnormal, 2^-149; the interval's own ends are rounded by 2^-24 |y|.  e covers all of it.
__device__ __forceinline__ uint32_t rotated_bf16x2(float a0, float b0, float a1, float b1, float c0, float s0, float c1, float s1) {
    constexpr float kRel = 1.2e-7f;   // over 2^-23
    constexpr float kAbs = 5.6e-45f;  // 2^-147
    const float q0 = b0 * s0, q1 = b1 * s1, y0 = fmaf(a0, c0, -q0), y1 = fmaf(a1, c1, -q1);
    const float e0 = fmaf(fabsf(y0) + fabsf(q0), kRel, kAbs), e1 = fmaf(fabsf(y1) + fabsf(q1), kRel, kAbs);
    uint32_t lo = pack_bf16(y0 - e0, y1 - e1);
    const uint32_t differ = lo ^ pack_bf16(y0 + e0, y1 + e1);
    if (differ & 0xFFFFu) lo = (lo & 0xFFFF0000u) | rotated_f64(a0, c0, b0, s0);
    if (differ >> 16) lo = (lo & 0xFFFFu) | rotated_f64(a1, c1, b1, s1) << 16;
    return lo;
}

// Four codes e4m3(fl64(y / s)) for y = a c - b sn rounded to binary64.  With y and q as above, y inv is off by
// 2^-24 |inv| (2 |y| + |q|), an interval's end rounded by 2^-24 |y inv|: within rel (|y| + |q|).  abs keeps values whose
// sign a subnormal y may have lost on both sides of zero.
__device__ __forceinline__ uint32_t e4m3_rotated(const float (&a)[4], const float (&b)[4], const float (&c)[4],
                                                 const float (&sn)[4], float sign, const Recip &r) {
    float lo[4], hi[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float q = sign * b[j] * sn[j], y = fmaf(a[j], c[j], -q);
        const float e = fmaf(fabsf(y) + fabsf(q), r.rel, r.abs);
        lo[j] = fmaf(y, r.inv, -e);
        hi[j] = fmaf(y, r.inv, e);
    }
    uint32_t code = e4m3x4(lo[0], lo[1], lo[2], lo[3]);
    if ((code ^ e4m3x4(hi[0], hi[1], hi[2], hi[3])) | r.odd) {
        code = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) code |= e4m3_rotated_f64(a[j], c[j], sign * b[j], sn[j], r.s) << (8 * j);
    }
    return code;
}
// Rotates a lane's dims in place, each value rounded once to bf16.
__device__ __forceinline__ void rotate_bf16(uint2 &x, uint2 &y, const float (&c)[4], const float (&s)[4]) {
    float a[4], b[4];
    unpack4(x, a);
    unpack4(y, b);
    x.x = rotated_bf16x2(a[0], b[0], a[1], b[1], c[0], s[0], c[1], s[1]);
    x.y = rotated_bf16x2(a[2], b[2], a[3], b[3], c[2], s[2], c[3], s[3]);
    y.x = rotated_bf16x2(b[0], -a[0], b[1], -a[1], c[0], s[0], c[1], s[1]);
    y.y = rotated_bf16x2(b[2], -a[2], b[3], -a[3], c[2], s[2], c[3], s[3]);
}

// Grid: [0, runs) x kv heads: runs of keys and values; the CTAs behind them:
// query rows, a warp each.
// Five CTAs an SM leave 48 registers a thread, of which 60 bytes are spilled.
__global__ void __launch_bounds__(kThreads, 5) paged_append_kernel(const __grid_constant__ PagedAppendArgs a, int runs) {
    const PagedSeqs &sq = a.seqs;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rot = a.rotary_dim, half = rot >> 1, ps = 1 << sq.page_shift;
    const LaneDims ld = lane_dims(lane, rot);
    __shared__ long long scan[33];
    __shared__ int found[4];
    __shared__ float edge[2][kWarps][kHeadDim];
    wait_for_previous_kernel();
    let_next_kernel_start();

    if ((int)blockIdx.x >= runs * a.num_kv_heads) {
        // ---- queries: a warp takes up to kQueryHeads heads of a row, which share its angles ----
        const int parts = (a.num_q_heads + kQueryHeads - 1) / kQueryHeads;
        const long long vec = (long long)(blockIdx.x - runs * a.num_kv_heads) * kWarps + warp;
        const int r = (int)(vec / parts), h0 = (int)(vec % parts) * kQueryHeads;
        if (r >= sq.num_tokens) return;
        const __nv_bfloat16 *src = a.q + (size_t)r * a.q_stride + h0 * kHeadDim;
        __nv_bfloat16 *dst = a.q_rot + ((size_t)r * a.num_q_heads + h0) * kHeadDim;
        const int heads = min(kQueryHeads, a.num_q_heads - h0);
        uint2 x[kQueryHeads], y[kQueryHeads];   // under way while the row's position is looked up
#pragma unroll
        for (int i = 0; i < kQueryHeads; ++i)
            if (i < heads) {
                x[i] = *reinterpret_cast<const uint2 *>(src + i * kHeadDim + ld.d0);
                y[i] = *reinterpret_cast<const uint2 *>(src + i * kHeadDim + ld.d1);
            }
        int bit;
        const SeqSpan q = span_of_row(sq, r, &bit);
        if (q.n == 0) return;
        float c[4], s[4];
        if (ld.i >= 0) load_angles(a.rope + (size_t)(q.ctx + r - q.row0) * half, ld.i, c, s);
#pragma unroll
        for (int i = 0; i < kQueryHeads; ++i) {
            if (i >= heads) break;
            if (ld.i >= 0) rotate_bf16(x[i], y[i], c, s);
            *reinterpret_cast<uint2 *>(dst + i * kHeadDim + ld.d0) = x[i];
            *reinterpret_cast<uint2 *>(dst + i * kHeadDim + ld.d1) = y[i];
        }
        return;
    }

    // ---- keys and values of one run ----
    const int run = blockIdx.x / a.num_kv_heads, h = blockIdx.x % a.num_kv_heads;
    int b, block;
    SeqSpan q;
    if (!find_run(sq, run, h == 0, scan, found, &b, &block, &q)) return;
    const int page = sq.table[(size_t)b * sq.table_stride + block];
    if (page < 0 || page >= sq.num_pages) {
        if (tid == 0) atomicOr(sq.err, HD_DEVERR_PAGE);
        return;
    }
    const int p0 = max(q.ctx, block << sq.page_shift), p1 = min(q.ctx + q.n, (block + 1) << sq.page_shift);
    const bool fp8 = a.kv_type == KV_FP8;
    const Recip kr = recip_of(fp8 ? a.k_scale[h] : 1.f), vr = recip_of(fp8 ? a.v_scale[h] : 1.f);
    uint32_t lo[4], hi[4];   // of the keys' dims: bf16 pairs, or f16 pairs, which hold every E4M3 value
    const uint32_t inf = fp8 ? 0x7C007C00u : 0x7F807F80u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        lo[j] = inf;
        hi[j] = inf | 0x80008000u;
    }
    for (int p = p0 + warp; p < p1; p += kWarps) {
        const int r = q.row0 + p - q.ctx;
        const __nv_bfloat16 *ksrc = a.k + (size_t)r * a.k_stride + h * kHeadDim;
        const __nv_bfloat16 *vsrc = a.v + (size_t)r * a.v_stride + h * kHeadDim;
        const size_t o = (size_t)page * a.page_stride + ((size_t)h * ps + (p & (ps - 1))) * kHeadDim;
        uint2 x = *reinterpret_cast<const uint2 *>(ksrc + ld.d0), y = *reinterpret_cast<const uint2 *>(ksrc + ld.d1);
        const uint4 v = *reinterpret_cast<const uint4 *>(vsrc + 8 * lane);
        float c[4], s[4];
        if (ld.i >= 0) load_angles(a.rope + (size_t)p * half, ld.i, c, s);
        if (fp8) {
            float u[4], w[4], f[8];
            unpack4(x, u);
            unpack4(y, w);
            uint32_t cx, cy;
            if (ld.i >= 0) {
                cx = e4m3_rotated(u, w, c, s, 1.f, kr);
                cy = e4m3_rotated(w, u, c, s, -1.f, kr);
            } else {
                cx = e4m3_plain(u, kr);
                cy = e4m3_plain(w, kr);
            }
            uint8_t *kd = static_cast<uint8_t *>(a.cache_k) + o;
            *reinterpret_cast<uint32_t *>(kd + ld.d0) = cx;
            *reinterpret_cast<uint32_t *>(kd + ld.d1) = cy;
            unpack_bf16x8(v, f);
            const float v0[4] = {f[0], f[1], f[2], f[3]}, v1[4] = {f[4], f[5], f[6], f[7]};
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.cache_v) + o + 8 * lane) =
                make_uint2(e4m3_plain(v0, vr), e4m3_plain(v1, vr));
            widen2<false>(lo[0], hi[0], e4m3x2_to_f16x2(cx & 0xFFFFu));
            widen2<false>(lo[1], hi[1], e4m3x2_to_f16x2(cx >> 16));
            widen2<false>(lo[2], hi[2], e4m3x2_to_f16x2(cy & 0xFFFFu));
            widen2<false>(lo[3], hi[3], e4m3x2_to_f16x2(cy >> 16));
        } else {
            if (ld.i >= 0) rotate_bf16(x, y, c, s);
            __nv_bfloat16 *kd = static_cast<__nv_bfloat16 *>(a.cache_k) + o;
            *reinterpret_cast<uint2 *>(kd + ld.d0) = x;
            *reinterpret_cast<uint2 *>(kd + ld.d1) = y;
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.cache_v) + o + 8 * lane) = v;
            widen2<true>(lo[0], hi[0], x.x);
            widen2<true>(lo[1], hi[1], x.y);
            widen2<true>(lo[2], hi[2], y.x);
            widen2<true>(lo[3], hi[3], y.y);
        }
    }
    if (a.bounds) store_bounds(a, page, h, fp8, (p0 & (ps - 1)) == 0, ld, lo, hi, edge);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs &a, cudaStream_t s) {
    const PagedSeqs &q = a.seqs;
    const long long runs = max_runs(q);
    const long long parts = (a.num_q_heads + kQueryHeads - 1) / kQueryHeads;
    const long long qctas = a.q ? ((long long)q.num_tokens * parts + kWarps - 1) / kWarps : 0;
    const long long grid = runs * a.num_kv_heads + qctas;
    if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
    return launch_overlapping(paged_append_kernel, dim3((unsigned)grid), kThreads, 0, 1, s, a, (int)runs);
}

}  // namespace hd
