// Pieces that the calls which write entries of a paged cache share: E4M3 codes
// of given values, a lane's dims of a row, a page's key bounds, and the run of
// new tokens that a CTA owns.
#pragma once

#include <cuda_fp8.h>

#include "e4m3.cuh"
#include "paged_sched.cuh"
#include "rope_round.cuh"

namespace hd {
namespace {

constexpr int kEntryThreads = 256;
constexpr int kEntryWarps = kEntryThreads / 32;

// A binary64 path is a call: inlined at every use it makes the kernels wait for their instructions.
__device__ __noinline__ uint32_t e4m3_rotated_f64(float a, float c, float b, float sn, float s) {
    const double y = __dsub_rn(__dmul_rn((double)a, (double)c), __dmul_rn((double)b, (double)sn));
    return e4m3_from_f64(__ddiv_rn(y, (double)s));
}

// A scale's reciprocal, and the bounds that go with it.
struct Recip {
    float s, inv;   // inv = RN(1 / s)
    float rel, abs;
    uint32_t odd;   // all ones: the reciprocal is no normal number
};
__device__ __forceinline__ Recip recip_of(float s) {
    Recip r;
    r.s = s;
    r.inv = 1.f / s;
    const float m = fabsf(r.inv);
    r.odd = m > 1.2e-38f && m < 3e38f ? 0u : 0xFFFFFFFFu;
    r.rel = 2.4e-7f * m;   // over 2^-22 |1 / s|
    r.abs = fmaf(m, 7.2e-43f, 7.2e-43f);
    return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float x0, float x1, float x2, float x3) {
    const uint32_t l = __nv_cvt_float2_to_fp8x2(make_float2(x0, x1), __NV_SATFINITE, __NV_E4M3);
    const uint32_t h = __nv_cvt_float2_to_fp8x2(make_float2(x2, x3), __NV_SATFINITE, __NV_E4M3);
    return l | h << 16;
}

// Four codes e4m3(fl64(a / s)).  a inv carries a's sign to the last.
__device__ __forceinline__ uint32_t e4m3_plain(const float (&a)[4], const Recip &r) {
    float lo[4], hi[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float e = fabsf(a[j]) * r.rel;
        lo[j] = fmaf(a[j], r.inv, -e);
        hi[j] = fmaf(a[j], r.inv, e);
    }
    uint32_t code = e4m3x4(lo[0], lo[1], lo[2], lo[3]);
    if ((code ^ e4m3x4(hi[0], hi[1], hi[2], hi[3])) | r.odd) {
        code = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) code |= e4m3_rotated_f64(a[j], 1.f, 0.f, 0.f, r.s) << (8 * j);
    }
    return code;
}

// Elementwise minimum and maximum of two bf16 or two f16, numbers before NaN.
template <bool BF16>
__device__ __forceinline__ void widen2(uint32_t &lo, uint32_t &hi, uint32_t x) {
    if (BF16) {
        asm("min.bf16x2 %0, %0, %1;" : "+r"(lo) : "r"(x));
        asm("max.bf16x2 %0, %0, %1;" : "+r"(hi) : "r"(x));
    } else {
        asm("min.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(x));
        asm("max.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(x));
    }
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t x;
    asm("{.reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t;}" : "=r"(x) : "r"(codes));
    return x;
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
__device__ __forceinline__ void load_angles(const float2 *cs, int i, float (&c)[4], float (&s)[4]) {
    const float4 u = __ldg(reinterpret_cast<const float4 *>(cs + i)), v = __ldg(reinterpret_cast<const float4 *>(cs + i + 2));
    c[0] = u.x; s[0] = u.y; c[1] = u.z; s[1] = u.w;
    c[2] = v.x; s[2] = v.y; c[3] = v.z; s[3] = v.w;
}

// The run of keys and values number `run` of a call: the new tokens of sequence b in its block `block`, by every thread of
// a CTA of kEntryThreads.  False: no such run, or a sequence that cannot be served (flagged by the CTA with `report`).
// `scan`: 33 words, `found`: 2, of shared memory.
__device__ __forceinline__ bool find_run(const PagedSeqs &sq, int run, bool report, long long *scan, int *found, int *seq,
                                         int *blk, SeqSpan *span) {
    const int tid = threadIdx.x;
    int b = run, block = 0, bit = 0;
    if (sq.offsets) {
        const int per = (sq.batch + kEntryThreads - 1) / kEntryThreads;
        const int b_lo = min(tid * per, sq.batch), b_hi = min(b_lo + per, sq.batch);
        long long mine = 0, total;
        int bad = 0;
        for (int i = b_lo; i < b_hi; ++i) {
            const SeqSpan q = seq_span(sq, i, &bit);
            bad |= bit;
            if (q.n) mine += ((q.ctx + q.n - 1) >> sq.page_shift) - (q.ctx >> sq.page_shift) + 1;
        }
        if (bad && run == 0 && report) atomicOr(sq.err, bad);
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
        if (b < 0) return false;
        block = found[1];
    }
    const SeqSpan q = seq_span(sq, b, &bit);
    if (q.n == 0) {
        if (bit && !sq.offsets && report && tid == 0) atomicOr(sq.err, bit);
        return false;
    }
    *seq = b;
    *blk = sq.offsets ? block : q.ctx >> sq.page_shift;
    *span = q;
    return true;
}

// The bounds of a page's kv head after a run: the warps' minima and maxima `lo` / `hi` over its keys' codes or bf16 values,
// merged through `edge`, and with what the page had unless the run starts it anew (`fresh`).  Every thread of the CTA.
__device__ __forceinline__ void store_bounds(const PagedAppendArgs &a, int page, int h, bool fp8, bool fresh, const LaneDims &ld,
                                             const uint32_t (&lo)[4], const uint32_t (&hi)[4],
                                             float (&edge)[2][kEntryWarps][kHeadDim]) {
    const int tid = threadIdx.x, warp = tid >> 5;
    auto pair = [&](uint32_t w) {
        return fp8 ? __half22float2(*reinterpret_cast<const __half2 *>(&w))
                   : make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    };
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int d = (j < 2 ? ld.d0 : ld.d1) + 2 * (j & 1);
        *reinterpret_cast<float2 *>(&edge[0][warp][d]) = pair(lo[j]);
        *reinterpret_cast<float2 *>(&edge[1][warp][d]) = pair(hi[j]);
    }
    __syncthreads();
    __nv_bfloat16 *bd = a.bounds + ((size_t)page * a.num_kv_heads + h) * 2 * kHeadDim;
    for (int d = tid; d < kHeadDim; d += kEntryThreads) {
        float l = edge[0][0][d], m = edge[1][0][d];
#pragma unroll
        for (int w = 1; w < kEntryWarps; ++w) {
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

// Grid of runs of a call: a sequence of n tokens touches at most (n - 1) / page + 2 pages, one of one token exactly one.
inline long long max_runs(const PagedSeqs &q) {
    return q.offsets ? ((long long)q.num_tokens >> q.page_shift) + 2LL * q.batch : q.batch;
}

}  // namespace
}  // namespace hd
