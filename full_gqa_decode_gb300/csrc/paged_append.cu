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
// The written key is the exact rotation rounded once (rope_round.cuh for
// bf16).  An E4M3 entry is e4m3(y / scale): binary32 with an error bound,
// binary64 next to a rounding border -- GB300 runs binary64 at a sixtieth of
// the binary32 rate, and evaluating every key there would bound the call.
#include <cuda_fp8.h>

#include "e4m3.cuh"
#include "paged_sched.cuh"
#include "rope_round.cuh"

namespace hd {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kQueryHeads = 4;   // heads of a row that one warp rotates

// The binary64 paths are calls: inlined at every use they make the kernel wait for its instructions (append of 9026
// tokens at 16 heads: 94 us inlined, 87 us so).
__device__ __noinline__ uint8_t e4m3_rotated_f64(float a, float c, float b, float sn, float s) {
    const double y = __dsub_rn(__dmul_rn((double)a, (double)c), __dmul_rn((double)b, (double)sn));
    return e4m3_from_f64(__ddiv_rn(y, (double)s));
}
__device__ __noinline__ float rotated_f64(float a, float c, float b, float s) {
    return f64_to_bf16_value(__dsub_rn(__dmul_rn((double)a, (double)c), __dmul_rn((double)b, (double)s)));
}

// e4m3(fl64(y / s)) for y = a c - b sn (the exact rotation, rounded once to
// binary64), bit for bit.  In binary32: q = RN(b sn), y32 = fma(a, c, -q) with
// |y32 - y| <= 2^-24 (|y32| + |q|), and t = RN(y32 / s) adds 2^-24 |t|.  In
// units of t's E4M3 quantum that sum is at most `err` (1% over it for the
// second-order terms).  The code is that of t unless t lies within err of a
// midpoint, its sign is in doubt, or it is no ordinary number -- then binary64
// decides.  inv = |1 / s|.  (c, sn) = (1, 0): the value a itself.
__device__ __forceinline__ uint8_t e4m3_rotated(float a, float c, float b, float sn, float s, float inv) {
    const float q = b * sn, y = fmaf(a, c, -q);
    const float t = __fdiv_rn(y, s), mag = fabsf(t);
    if (mag < 1e30f && mag > 1e-30f && fabsf(y) > 1e-30f) {
        const int e = max((int)(__float_as_uint(mag) >> 23) - 127, -6);
        const float per = __uint_as_float((uint32_t)(127 + 3 - e) << 23);   // 1 / quantum
        const float u = mag * per;                                           // exact
        const float err = 6.02e-8f * (mag + (fabsf(y) + fabsf(q)) * inv) * per;
        if (fabsf(u - truncf(u) - 0.5f) > err && u > err) return __nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
    }
    return e4m3_rotated_f64(a, c, b, sn, s);
}

// A lane's eight dims of a row: two runs of four, at d0 and d1.
struct LaneDims {
    int d0, d1, i;   // i: first rotary pair (-1: past the rotation)
};
__device__ __forceinline__ LaneDims lane_dims(int lane, int rot) {
    const int half = rot >> 1;
    if (4 * lane < half) return {4 * lane, 4 * lane + half, 4 * lane};
    const int d = rot + 8 * (lane - half / 4);
    return {d, d + 4, -1};
}
__device__ __forceinline__ void unpack4(uint2 w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x << 16);
    x[1] = __uint_as_float(w.x & 0xFFFF0000u);
    x[2] = __uint_as_float(w.y << 16);
    x[3] = __uint_as_float(w.y & 0xFFFF0000u);
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float (&x)[4]) { unpack4(*reinterpret_cast<const uint2 *>(p), x); }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float (&x)[4]) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}
__device__ __forceinline__ void load_angles(const float2 *cs, int i, float (&c)[4], float (&s)[4]) {
    const float4 u = __ldg(reinterpret_cast<const float4 *>(cs + i)), v = __ldg(reinterpret_cast<const float4 *>(cs + i + 2));
    c[0] = u.x; s[0] = u.y; c[1] = u.z; s[1] = u.w;
    c[2] = v.x; s[2] = v.y; c[3] = v.z; s[3] = v.w;
}

// Rotates a lane's dims in place, each value rounded once to bf16.
__device__ __forceinline__ void rotate_bf16(float (&x)[4], float (&y)[4], const float (&c)[4], const float (&s)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float a = x[j], b = y[j];
        float u, v;
        const bool sure = rotated_bf16_sure(a, c[j], b, s[j], &u) & rotated_bf16_sure(b, c[j], -a, s[j], &v);
        if (!sure) {
            u = rotated_f64(a, c[j], b, s[j]);
            v = rotated_f64(b, c[j], -a, s[j]);
        }
        x[j] = u;
        y[j] = v;
    }
}

// Grid: [0, runs) x kv heads: runs of keys and values; the CTAs behind them:
// query rows, a warp each.
__global__ void __launch_bounds__(kThreads, 4) paged_append_kernel(const __grid_constant__ PagedAppendArgs a, int runs) {
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
            if (ld.i >= 0) {
                float u[4], v[4];
                unpack4(x[i], u);
                unpack4(y[i], v);
                rotate_bf16(u, v, c, s);
                x[i] = make_uint2(pack_bf16(u[0], u[1]), pack_bf16(u[2], u[3]));
                y[i] = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
            }
            *reinterpret_cast<uint2 *>(dst + i * kHeadDim + ld.d0) = x[i];
            *reinterpret_cast<uint2 *>(dst + i * kHeadDim + ld.d1) = y[i];
        }
        return;
    }

    // ---- keys and values of one run ----
    const int run = blockIdx.x / a.num_kv_heads, h = blockIdx.x % a.num_kv_heads;
    int b = run, block = 0, bit = 0;
    if (sq.offsets) {
        const int per = (sq.batch + kThreads - 1) / kThreads;
        const int b_lo = min(tid * per, sq.batch), b_hi = min(b_lo + per, sq.batch);
        long long mine = 0, total;
        int bad = 0;
        for (int i = b_lo; i < b_hi; ++i) {
            const SeqSpan q = seq_span(sq, i, &bit);
            bad |= bit;
            if (q.n) mine += ((q.ctx + q.n - 1) >> sq.page_shift) - (q.ctx >> sq.page_shift) + 1;
        }
        if (bad && run == 0 && h == 0) atomicOr(sq.err, bad);
        if (tid == 0) found[0] = -1;
        const long long before = block_prefix(mine, scan, &total);
        if (before <= run && run < before + mine) {
            long long rem = run - before;
            for (int i = b_lo; i < b_hi; ++i) {
                const SeqSpan q = seq_span(sq, i, &bit);
                if (!q.n) continue;
                const int nb = ((q.ctx + q.n - 1) >> sq.page_shift) - (q.ctx >> sq.page_shift) + 1;
                if (rem < nb) {
                    found[0] = i;
                    found[1] = (q.ctx >> sq.page_shift) + (int)rem;
                    break;
                }
                rem -= nb;
            }
        }
        __syncthreads();
        b = found[0];
        if (b < 0) return;
        block = found[1];
    }
    const SeqSpan q = seq_span(sq, b, &bit);
    if (q.n == 0) {
        if (bit && !sq.offsets && h == 0 && tid == 0) atomicOr(sq.err, bit);
        return;
    }
    if (!sq.offsets) block = q.ctx >> sq.page_shift;
    const int page = sq.table[(size_t)b * sq.table_stride + block];
    if (page < 0 || page >= sq.num_pages) {
        if (tid == 0) atomicOr(sq.err, HD_DEVERR_PAGE);
        return;
    }
    const int p0 = max(q.ctx, block << sq.page_shift), p1 = min(q.ctx + q.n, (block + 1) << sq.page_shift);
    const bool fp8 = a.kv_type == KV_FP8;
    const float ks = fp8 ? a.k_scale[h] : 1.f, vs = fp8 ? a.v_scale[h] : 1.f;
    const float kinv = fp8 ? fabsf(1.f / ks) : 1.f, vinv = fp8 ? fabsf(1.f / vs) : 1.f;
    float lo[8], hi[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        lo[j] = INFINITY;
        hi[j] = -INFINITY;
    }
    for (int p = p0 + warp; p < p1; p += kWarps) {
        const int r = q.row0 + p - q.ctx;
        const __nv_bfloat16 *ksrc = a.k + (size_t)r * a.k_stride + h * kHeadDim;
        const __nv_bfloat16 *vsrc = a.v + (size_t)r * a.v_stride + h * kHeadDim;
        const size_t o = (size_t)page * a.page_stride + ((size_t)h * ps + (p & (ps - 1))) * kHeadDim;
        float x[4], y[4], c[4], s[4];
        load4(ksrc + ld.d0, x);
        load4(ksrc + ld.d1, y);
        const uint4 v = *reinterpret_cast<const uint4 *>(vsrc + 8 * lane);
        if (ld.i >= 0) load_angles(a.rope + (size_t)p * half, ld.i, c, s);
        if (fp8) {
            uint32_t cx = 0, cy = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float u = x[j], w = y[j];
                uint8_t kx, ky;
                if (ld.i >= 0) {
                    kx = e4m3_rotated(u, c[j], w, s[j], ks, kinv);
                    ky = e4m3_rotated(w, c[j], -u, s[j], ks, kinv);
                } else {
                    kx = e4m3_rotated(u, 1.f, 0.f, 0.f, ks, kinv);
                    ky = e4m3_rotated(w, 1.f, 0.f, 0.f, ks, kinv);
                }
                cx |= (uint32_t)kx << (8 * j);
                cy |= (uint32_t)ky << (8 * j);
                x[j] = e4m3_to_f32(kx);
                y[j] = e4m3_to_f32(ky);
            }
            uint8_t *kd = static_cast<uint8_t *>(a.cache_k) + o;
            *reinterpret_cast<uint32_t *>(kd + ld.d0) = cx;
            *reinterpret_cast<uint32_t *>(kd + ld.d1) = cy;
            float f[8];
            unpack_bf16x8(v, f);
            uint32_t w0 = 0, w1 = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w0 |= (uint32_t)e4m3_rotated(f[j], 1.f, 0.f, 0.f, vs, vinv) << (8 * j);
                w1 |= (uint32_t)e4m3_rotated(f[4 + j], 1.f, 0.f, 0.f, vs, vinv) << (8 * j);
            }
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.cache_v) + o + 8 * lane) = make_uint2(w0, w1);
        } else {
            if (ld.i >= 0) rotate_bf16(x, y, c, s);
            __nv_bfloat16 *kd = static_cast<__nv_bfloat16 *>(a.cache_k) + o;
            store4(kd + ld.d0, x);
            store4(kd + ld.d1, y);
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.cache_v) + o + 8 * lane) = v;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            lo[j] = fminf(lo[j], x[j]);
            hi[j] = fmaxf(hi[j], x[j]);
            lo[4 + j] = fminf(lo[4 + j], y[j]);
            hi[4 + j] = fmaxf(hi[4 + j], y[j]);
        }
    }
    if (!a.bounds) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        edge[0][warp][ld.d0 + j] = lo[j];
        edge[0][warp][ld.d1 + j] = lo[4 + j];
        edge[1][warp][ld.d0 + j] = hi[j];
        edge[1][warp][ld.d1 + j] = hi[4 + j];
    }
    __syncthreads();
    __nv_bfloat16 *bd = a.bounds + ((size_t)page * a.num_kv_heads + h) * 2 * kHeadDim;
    const bool fresh = (p0 & (ps - 1)) == 0;
    for (int d = tid; d < kHeadDim; d += kThreads) {
        float l = edge[0][0][d], m = edge[1][0][d];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            l = fminf(l, edge[0][w][d]);
            m = fmaxf(m, edge[1][w][d]);
        }
        if (!fresh) {
            l = fminf(l, __bfloat162float(bd[d]));
            m = fmaxf(m, __bfloat162float(bd[kHeadDim + d]));
        }
        bd[d] = __float2bfloat16_rn(l);             // exact: bf16 keys or E4M3 code values
        bd[kHeadDim + d] = __float2bfloat16_rn(m);
    }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs &a, cudaStream_t s) {
    const PagedSeqs &q = a.seqs;
    // A sequence of n tokens touches at most (n - 1) / page + 2 pages, one of one token exactly one.
    const long long runs = q.offsets ? ((long long)q.num_tokens >> q.page_shift) + 2LL * q.batch : q.batch;
    const long long parts = (a.num_q_heads + kQueryHeads - 1) / kQueryHeads;
    const long long qctas = a.q ? ((long long)q.num_tokens * parts + kWarps - 1) / kWarps : 0;
    const long long grid = runs * a.num_kv_heads + qctas;
    if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
    return launch_overlapping(paged_append_kernel, dim3((unsigned)grid), kThreads, 0, 1, s, a, (int)runs);
}

}  // namespace hd
