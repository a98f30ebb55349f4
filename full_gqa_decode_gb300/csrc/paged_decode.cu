// Attention of few query rows per kv head over a paged cache: single-token
// decode, a few drafted tokens, and decode over selected pages.
//
// Each item (sequence, up to eight query rows = heads x tokens, kv head)
// streams its visible keys once: HBM bounds it, so the arithmetic only has to
// keep out of the way.  One persistent CTA per SM runs a ring of six 32 KiB
// stages (32 bf16 or 64 E4M3 keys of K and V) on across items.  One producer
// warp looks the pages up and issues one 5-D TMA copy per page run and stage
// half -- the box takes all 256 dims as 128-byte column groups, so a stage is
// two copies for pages of at least a stage's keys, four to eight otherwise.
// Eight consumer warps take 16 keys each; the warps of a stage (two, or four
// with E4M3) form a team and the teams take stages in turn, so a warp's chain of
// dependent MMAs and shuffles overlaps the other teams' and not only its own
// stage's copies.  The work is cut evenly over the CTAs (paged_sched.cuh).
// Measured: 64 sequences of 512 to 32768 keys 336 us (6.9 TB/s of keys and values);
// 256 of 512 to 8192 at group 8 over E4M3 pages 201 us (5.8 TB/s, bound by the warps'
// conversions, MMAs and shuffles); one sequence at 4096 12 us, all latency.
//
// Per 16 keys, on mma.sync m16n8k16 with an online softmax in log2 units:
//     S^T = K Q^T   keys on M, the rows on N: q takes two registers a k-step
//     O^T += V^T P^T   dims on M; P^T is the scores' fragment transposed
// Rotated queries enter the products in bf16 as they come.  With an E4M3 cache
// codes convert exactly to f16, and a row's q is scaled by the power of two that
// brings its largest value below 2, so that f16 holds it: values below 2^-14 of
// that lose bits under 2^-25 of the largest, less than the fp32 sum of the
// products does.  With bf16 pages P enters the second product in two bf16 parts,
// the rounded weight and what the rounding left (2^-16 of the weight remain): in
// one part alone its rounding adds as much to the error as the output's own
// (2.2e-3 against 1.7e-3 of the output, root mean square), and the second
// product of a fragment is nearly free (one sequence at 4096 12.7 and 12.9 us, 64
// sequences 337 and 336 us).  With E4M3 pages one f16 part is enough (2^-11 of a
// weight); f16 weights are taken 2^15 times as large, which the division by their
// sum undoes, so that small ones stay clear of f16's subnormals.  Sums and maxima
// stay in fp32.
//
// Scored rows (attn_paged_scored) are an instance of the same kernel: their tiles
// range over what any of their rows sees, and a score is capped and biased
// between its product and its weight, a few instructions in the shadow of the
// reads.  Measured: one sequence at 4096 capped 12.9 us, 64 sequences of 512 to
// 32768 capped 333 us (7.0 TB/s), 256 of 512 to 8192 at group 8 over E4M3 pages
// with a bias by distance 202 us (5.8 TB/s; 32 bytes a thread spilled).
#include "paged_rows.cuh"

namespace hd {
namespace {

constexpr int kRing = 6;                        // stages of 32 KiB
// Barriers of landed stages: two rounds of the ring, so that a barrier always serves the same team, which cannot
// take a round for the one before it (a parity tells only neighbouring rounds apart).
constexpr int kFulls = 2 * kRing;
constexpr int kWarpKeys = 16;                   // keys a warp takes at a time
constexpr int kWarps = 8;                       // consumer warps
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kRowPad = kHeadDim + 4;           // floats between rows of a merge buffer: fragment stores hit all banks
constexpr int kBufFloats = kDecodeRows * kRowPad;
constexpr int kBufs = kWarps / 2;
// Shared memory: ring | merge buffers | row maxima and sums | barriers | scan and flags | page runs of a stage.
constexpr int kBufOff = kRing * kStageBytes;
constexpr int kMlOff = kBufOff + kBufs * kBufFloats * 4;
constexpr int kBarOff = kMlOff + 2 * (kWarps + 1) * kDecodeRows * 4;
constexpr int kMiscOff = kBarOff + (kFulls + kRing) * 8;
constexpr int kPosOff = kMiscOff + 48;          // [kRing][4] positions of a stage's page runs (selected blocks)
constexpr int kSmemBytes = kPosOff + kRing * 4 * 4;
static_assert(kSmemBytes <= 227 * 1024, "one CTA per SM");
static_assert(kDecodeCtasPerSm == 1, "the partials' workspace counts one CTA per SM");

__host__ __device__ constexpr int stage_shift(int kv) { return kv == KV_FP8 ? 6 : 5; }
// Warps of a stage's team, and the shortest share of a CTA in stages.
__host__ __device__ constexpr int team_warps(int kv) { return (1 << stage_shift(kv)) / kWarpKeys; }
__host__ __device__ constexpr int min_units(int kv) { return kv == KV_FP8 ? 2 : 4; }

// Items of up to this many stages are not cut in short calls: an item's pieces and their merge cost about 5 us, the
// time of some 20 stages (512-key windows of 64 sequences: 23.2 us cut evenly, 18.1 us whole).
constexpr int kSnap = 40;

// A tile of new tokens of one sequence.
struct Tile {
    int t0, nt;       // tokens
    int lo, hi;       // visible positions [lo, hi) of any of them (SPARSE: hi only)
    int u0, units;    // stages
};

template <int KV, bool SPARSE>
__device__ __forceinline__ int tile_tokens(const PagedAttnArgs &a) {
    return SPARSE ? 1 : kDecodeRows >> a.group_shift;
}

template <int KV, bool SPARSE, bool SCORED>
__device__ __forceinline__ Tile make_tile(const PagedAttnArgs &a, const SeqSpan &q, int tile) {
    constexpr int kShift = stage_shift(KV), kKeys = 1 << kShift;
    const int tt = tile_tokens<KV, SPARSE>(a);
    if constexpr (SCORED) return scored_tile<Tile>(a, q, tile * tt, min(tt, q.n - tile * tt), kShift);
    Tile t;
    t.t0 = tile * tt;
    t.nt = min(tt, q.n - t.t0);
    t.hi = q.ctx + t.t0 + t.nt;
    if (SPARSE) {
        const int blocks = min(a.num_selected, ((t.hi - 1) >> a.seqs.page_shift) + 1);
        t.lo = 0;
        t.u0 = 0;
        t.units = (int)((((long long)blocks << a.seqs.page_shift) + kKeys - 1) >> kShift);
    } else {
        t.lo = a.window ? max(0, q.ctx + t.t0 - a.window + 1) : 0;
        t.u0 = t.lo >> kShift;
        t.units = ((t.hi + kKeys - 1) >> kShift) - t.u0;
    }
    return t;
}

// Where a CTA is in the list of items.
struct Cursor {
    int b, tile, h, off;   // off: stages of the item already passed
};

template <int KV, bool SPARSE>
__device__ __forceinline__ int num_tiles(const PagedAttnArgs &a, int n) {
    return SPARSE ? n : ((n << a.group_shift) + kDecodeRows - 1) / kDecodeRows;
}

// The item after (c, q): advances to the next kv head, tile or sequence.
template <int KV, bool SPARSE>
__device__ __forceinline__ void next_item(const PagedAttnArgs &a, Cursor &c, SeqSpan &q) {
    c.off = 0;
    if (++c.h < a.num_kv_heads) return;
    c.h = 0;
    if (++c.tile < num_tiles<KV, SPARSE>(a, q.n)) return;
    c.tile = 0;
    int bit;
    do {
        q = seq_span(a.seqs, ++c.b, &bit);
    } while (q.n == 0 && c.b + 1 < a.seqs.batch);
}

// Position of key `x` (a stage-aligned index into the item's keys) and the page holding it; -1: no page.
// SPARSE: x indexes the selected blocks' slots, and the position is huge past their end.
template <bool SPARSE>
__device__ __forceinline__ int key_position(const PagedAttnArgs &a, const int32_t *sel, const Tile &t, int x) {
    if (!SPARSE) return x;
    const int j = x >> a.seqs.page_shift, slot = x & ((1 << a.seqs.page_shift) - 1);
    const int blk = j < a.num_selected ? sel[j] : -1;
    if (blk < 0 || blk > ((t.hi - 1) >> a.seqs.page_shift)) return 0x40000000;
    return (blk << a.seqs.page_shift) + slot;
}

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory"); }
// Row of q / out / lse of row r of a tile.
__device__ __forceinline__ size_t query_row(const PagedAttnArgs &a, const SeqSpan &q, const Tile &t, int h, int r) {
    return (size_t)(q.row0 + t.t0 + (r >> a.group_shift)) * a.num_q_heads + (h << a.group_shift) + (r & (a.group - 1));
}

// ------------------------------------------------------------- consumers --
// One warp's 16 keys of a stage against the tile's rows.  `base`: byte offset
// of the warp's first key row in a stage half, `col`: bytes between its 128-byte
// column groups; key0: position of that key; [vlo, vhi): positions whose V may
// be read; first: position of the tile's first row; full: every row sees every
// key of the warp.

// What both cache types share: the softmax on S^T fragments (register r of
// lane (gid, t4): key gid + 8 (r / 2), row 2 t4 + r % 2), and the rows' state.
template <bool F16, bool SCORED>
struct DecodeRowsState {
    static constexpr float kLift = F16 ? 15.f : 0.f;
    float o[16][4];            // O^T: dims (two of tile mt) x rows 2 t4 (+ 1)
    float m_run[2], l_run[2];  // rows 2 t4 + e; l_run: this lane's keys
    RowSpan span[SCORED ? 2 : 1];     // their visible positions ..
    float slope[SCORED ? 2 : 1];      // .. and biases of a position's distance, log2 units

    // What a row's weights are taken against: its maximum less the lift.  Scored rows may have maxima beyond 2^23, where the
    // difference rounds: up, so that no weight is lifted by more (2^16, which rounding to nearest gave from 2^27 on, is
    // infinite in f16).
    __device__ static __forceinline__ float lifted(float m) { return SCORED && F16 ? __fadd_ru(m, -kLift) : m - kLift; }

    __device__ void init_rows() {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            m_run[e] = -INFINITY;
            l_run[e] = 0.f;
        }
#pragma unroll
        for (int mt = 0; mt < 16; ++mt)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[mt][j] = 0.f;
    }
    __device__ __forceinline__ void init_rule(const PagedAttnArgs &a, const SeqSpan &q, const Tile &t, int h, int lane) {
        if constexpr (SCORED) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 2 * (lane & 3) + e;
                span[e] = row_span(a, q, t.t0 + min(r >> a.group_shift, t.nt - 1));
                slope[e] = a.slopes ? a.slopes[(h << a.group_shift) + (r & (a.group - 1))] * kLog2e : 0.f;
            }
        }
    }
    // Scores (times scale[e], log2 units) to weights; returns the two P^T operands: keys 2 t4 (+ 1) and 8 + 2 t4
    // (+ 1) of row gid; bf16: and those of the weights' low parts.
    __device__ __forceinline__ void weigh(const PagedAttnArgs &a, const float (&s)[4], const float (&scale)[2], int key0,
                                          int first, bool full, int lane, uint32_t (&pb)[F16 ? 2 : 4]) {
        float p[4], alpha[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            bool v0 = true, v1 = true;
            const int k0 = key0 + (lane >> 2), pos = first + ((2 * (lane & 3) + e) >> a.group_shift);
            if (!full) {   // first: position of the tile's first row
                const int hi = SCORED ? span[e].hi : pos;
                const int lo = SCORED ? span[e].lo : a.window ? hi - a.window + 1 : 0;
                v0 = k0 >= lo && k0 <= hi;
                v1 = k0 + 8 >= lo && k0 + 8 <= hi;
            }
            // Scored rows: rounded as their maximum is, whatever is taken off behind.
            float x0 = SCORED ? __fmul_rn(s[e], scale[e]) : s[e] * scale[e], x1 = SCORED ? __fmul_rn(s[2 + e], scale[e]) : s[2 + e] * scale[e];
            if constexpr (SCORED) {
                if (a.cap != 0.f) {
                    x0 = capped(a, x0 * a.two_over_cap);
                    x1 = capped(a, x1 * a.two_over_cap);
                }
                const float far = (float)(k0 - pos);
                x0 = fmaf(-slope[e], fabsf(far), x0);
                x1 = fmaf(-slope[e], fabsf(far + 8.f), x1);
            }
            x0 = v0 ? x0 : -INFINITY;
            x1 = v1 ? x1 : -INFINITY;
            float mx = fmaxf(x0, x1);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float mn = fmaxf(m_run[e], mx);
            alpha[e] = mn == -INFINITY ? 1.f : fast_exp2(SCORED && F16 ? lifted(m_run[e]) - lifted(mn) : m_run[e] - mn);
            p[e] = v0 ? fast_exp2(x0 - lifted(mn)) : 0.f;
            p[2 + e] = v1 ? fast_exp2(x1 - lifted(mn)) : 0.f;
            l_run[e] = fmaf(l_run[e], alpha[e], p[e] + p[2 + e]);
            m_run[e] = mn;
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
            for (int mt = 0; mt < 16; ++mt) {
                o[mt][0] *= alpha[0];
                o[mt][1] *= alpha[1];
                o[mt][2] *= alpha[0];
                o[mt][3] *= alpha[1];
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t w = F16 ? pack_f16(p[2 * i], p[2 * i + 1]) : pack_bf16(p[2 * i], p[2 * i + 1]);
            pb[i] = movmatrix_trans(w);
            if constexpr (!F16)
                pb[2 + i] = movmatrix_trans(pack_bf16(p[2 * i] - __uint_as_float(w << 16),
                                                      p[2 * i + 1] - __uint_as_float(w & 0xFFFF0000u)));
        }
    }
    // Masks of the V values of keys 2 t4 (+ 1) and 8 + 2 t4 (+ 1): slots outside [vlo, vhi) may hold anything, and
    // 0 * NaN would reach every row.
    __device__ static __forceinline__ void value_masks(int key0, int vlo, int vhi, int lane, uint32_t &m01, uint32_t &m89) {
        const int k0 = key0 + 2 * (lane & 3);
        m01 = (k0 >= vlo && k0 < vhi ? 0x0000FFFFu : 0u) | (k0 + 1 >= vlo && k0 + 1 < vhi ? 0xFFFF0000u : 0u);
        m89 = (k0 + 8 >= vlo && k0 + 8 < vhi ? 0x0000FFFFu : 0u) | (k0 + 9 >= vlo && k0 + 9 < vhi ? 0xFFFF0000u : 0u);
    }
    // Rows' maxima and (whole warp's) sums, [warps][rows] each.
    __device__ void publish(float *mx, float *sums, int warp, int lane) const {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float l = l_run[e];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            if (lane < 4) {
                mx[warp * kDecodeRows + 2 * lane + e] = lifted(m_run[e]);
                sums[warp * kDecodeRows + 2 * lane + e] = l;
            }
        }
    }
};

// bf16 pages.  O^T tile mt: dims 16 mt + gid (+ 8).
template <bool SCORED>
struct DecodeBf16 : DecodeRowsState<false, SCORED> {
    using Rows = DecodeRowsState<false, SCORED>;
    using Rows::o;
    uint32_t qb[16][2];
    float scale[2];

    __device__ void init(const PagedAttnArgs &a, const SeqSpan &q, const Tile &t, int h, int lane) {
        const int gid = lane >> 2, t4 = lane & 3;
        const bool live = gid < t.nt << a.group_shift;
        const __nv_bfloat16 *src = a.q + query_row(a, q, t, h, gid) * kHeadDim + 2 * t4;
#pragma unroll
        for (int ks = 0; ks < 16; ++ks) {
            qb[ks][0] = live ? __ldg(reinterpret_cast<const uint32_t *>(src + 16 * ks)) : 0u;
            qb[ks][1] = live ? __ldg(reinterpret_cast<const uint32_t *>(src + 16 * ks + 8)) : 0u;
        }
        scale[0] = scale[1] = SCORED ? a.qscale : kQScale;
        Rows::init_rows();
        Rows::init_rule(a, q, t, h, lane);
    }

    __device__ void consume(const PagedAttnArgs &a, const uint8_t *kst, const uint8_t *vst, uint32_t base, uint32_t col,
                            int key0, int vlo, int vhi, int first, bool full, int lane) {
        const int lr = lane & 7;
        // K: matrices (keys 0-7, 8-15) x (dims 0-7, 8-15) of k-step ks.
        const uint32_t kb = smem_u32(kst) + base + (lr + (lane & 8)) * 128;
        const uint32_t kc = (uint32_t)lane >> 4;
        float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < 16; ++ks) {
            uint32_t x[4];
            ldsm_x4(kb + (ks >> 2) * col + ((((uint32_t)(2 * (ks & 3)) + kc) ^ lr) << 4), x[0], x[1], x[2], x[3]);
            mma_16816(ks & 1 ? s2 : s, x, qb[ks][0], qb[ks][1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += s2[i];
        uint32_t pb[4], m01, m89;
        Rows::weigh(a, s, scale, key0, first, full, lane, pb);
        if (full) {   // the masks fold away
            products(vst, base, col, lane, pb, 0xFFFFFFFFu, 0xFFFFFFFFu);
        } else {
            Rows::value_masks(key0, vlo, vhi, lane, m01, m89);
            products(vst, base, col, lane, pb, m01, m89);
        }
    }
    __device__ __forceinline__ void products(const uint8_t *vst, uint32_t base, uint32_t col, int lane,
                                             const uint32_t (&pb)[4], uint32_t m01, uint32_t m89) {
        const int lr = lane & 7;
        // V^T: matrices (dims 0-7, 8-15 of tile mt) x (keys 0-7, 8-15), transposed on the way.
        const uint32_t vb = smem_u32(vst) + base + (lr + ((lane & 16) >> 1)) * 128;
        const uint32_t vc = (uint32_t)(lane >> 3) & 1;
#pragma unroll
        for (int mt = 0; mt < 16; ++mt) {
            uint32_t x[4];
            ldsm_x4_trans(vb + (mt >> 2) * col + ((((uint32_t)(2 * (mt & 3)) + vc) ^ lr) << 4), x[0], x[1], x[2], x[3]);
            x[0] &= m01;
            x[1] &= m01;
            x[2] &= m89;
            x[3] &= m89;
            mma_16816(o[mt], x, pb[0], pb[1]);
            mma_16816(o[mt], x, pb[2], pb[3]);
        }
    }
    template <class F> __device__ void each(int lane, F f) {   // f(row, dim, value&)
        const int gid = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int mt = 0; mt < 16; ++mt) {
            f(2 * t4, 16 * mt + gid, o[mt][0]);
            f(2 * t4 + 1, 16 * mt + gid, o[mt][1]);
            f(2 * t4, 16 * mt + gid + 8, o[mt][2]);
            f(2 * t4 + 1, 16 * mt + gid + 8, o[mt][3]);
        }
    }
};

// E4M3 pages.  Lane (gid, t4) reads 16-byte chunks 2 t4 + (p & 1) + 8 (p >> 1)
// of key rows gid and gid + 8 at step p (eight lanes of a phase hit eight
// different chunks); q's columns are held in the same order of dims, which
// leaves every dot product as it is.  O^T tile mt: dims 128 (mt / 8) + 16 gid +
// 2 (mt % 8) (+ 1).
template <bool SCORED>
struct DecodeE4m3 : DecodeRowsState<true, SCORED> {
    using Rows = DecodeRowsState<true, SCORED>;
    using Rows::o;
    uint32_t qb[16][2];
    float scale[2];

    __device__ void init(const PagedAttnArgs &a, const SeqSpan &q, const Tile &t, int h, int lane) {
        const int gid = lane >> 2, t4 = lane & 3;
        const bool live = gid < t.nt << a.group_shift;
        const __nv_bfloat16 *src = a.q + query_row(a, q, t, h, gid) * kHeadDim;
        uint32_t top = 0;
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int d = 16 * (2 * t4 + (p & 1) + 8 * (p >> 1)) + 4 * j;
                const uint2 w = live ? __ldg(reinterpret_cast<const uint2 *>(src + d)) : make_uint2(0u, 0u);
                qb[4 * p + j][0] = w.x;
                qb[4 * p + j][1] = w.y;
                const uint2 m = make_uint2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu);
                top = max(top, max(max(m.x & 0xFFFFu, m.x >> 16), max(m.y & 0xFFFFu, m.y >> 16)));
            }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = min(max((int)(top >> 7), 1), 253);               // exponent field of the row's largest value
        const float down = __uint_as_float((uint32_t)(254 - ex) << 23);  // 2^(127 - ex)
        const float up = __uint_as_float((uint32_t)ex << 23);
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                qb[i][j] = pack_f16(__uint_as_float(qb[i][j] << 16) * down, __uint_as_float(qb[i][j] & 0xFFFF0000u) * down);
#pragma unroll
        for (int e = 0; e < 2; ++e) scale[e] = __shfl_sync(0xffffffffu, up, 4 * (2 * t4 + e)) * (a.k_scale[h] * (SCORED ? a.qscale : kQScale));
        Rows::init_rows();
        Rows::init_rule(a, q, t, h, lane);
    }

    __device__ void consume(const PagedAttnArgs &a, const uint8_t *kst, const uint8_t *vst, uint32_t base, uint32_t col,
                            int key0, int vlo, int vhi, int first, bool full, int lane) {
        const int gid = lane >> 2, t4 = lane & 3;
        auto at = [&](int r, int c) { return base + (uint32_t)(c >> 3) * col + r * 128 + (((c & 7) ^ (r & 7)) << 4); };
        float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int chunk = 2 * t4 + (p & 1) + 8 * (p >> 1);
            const uint4 ka = *reinterpret_cast<const uint4 *>(kst + at(gid, chunk));
            const uint4 kb = *reinterpret_cast<const uint4 *>(kst + at(gid + 8, chunk));
            const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t x[4] = {e4m3x2_to_f16x2((uint16_t)(wa[j] & 0xFFFFu)), e4m3x2_to_f16x2((uint16_t)(wb[j] & 0xFFFFu)),
                                       e4m3x2_to_f16x2((uint16_t)(wa[j] >> 16)), e4m3x2_to_f16x2((uint16_t)(wb[j] >> 16))};
                mma_16816_f16(j & 1 ? s2 : s, x, qb[4 * p + j][0], qb[4 * p + j][1]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += s2[i];
        uint32_t pb[2], m01, m89;
        Rows::weigh(a, s, scale, key0, first, full, lane, pb);
        if (full) {   // the masks fold away
            products(vst, base, col, lane, pb, 0xFFFFFFFFu, 0xFFFFFFFFu);
        } else {
            Rows::value_masks(key0, vlo, vhi, lane, m01, m89);
            products(vst, base, col, lane, pb, m01, m89);
        }
    }
    __device__ __forceinline__ void products(const uint8_t *vst, uint32_t base, uint32_t col, int lane,
                                             const uint32_t (&pb)[2], uint32_t m01, uint32_t m89) {
        const int gid = lane >> 2, t4 = lane & 3;
        auto at = [&](int r, int c) { return base + (uint32_t)(c >> 3) * col + r * 128 + (((c & 7) ^ (r & 7)) << 4); };
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int chunk = 8 * half + gid;
            const uint4 v0 = *reinterpret_cast<const uint4 *>(vst + at(2 * t4, chunk));
            const uint4 v1 = *reinterpret_cast<const uint4 *>(vst + at(2 * t4 + 1, chunk));
            const uint4 v8 = *reinterpret_cast<const uint4 *>(vst + at(2 * t4 + 8, chunk));
            const uint4 v9 = *reinterpret_cast<const uint4 *>(vst + at(2 * t4 + 9, chunk));
            const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
            const uint32_t w8[4] = {v8.x, v8.y, v8.z, v8.w}, w9[4] = {v9.x, v9.y, v9.z, v9.w};
#pragma unroll
            for (int w = 0; w < 4; ++w)
#pragma unroll
                for (int q = 0; q < 2; ++q) {   // dims 4 w + 2 q (row gid) and 4 w + 2 q + 1 (row gid + 8)
                    const uint32_t sel = q ? 0x7362u : 0x5140u;
                    const uint32_t x01 = __byte_perm(w0[w], w1[w], sel), x89 = __byte_perm(w8[w], w9[w], sel);
                    const uint32_t x[4] = {e4m3x2_to_f16x2((uint16_t)(x01 & 0xFFFFu)) & m01, e4m3x2_to_f16x2((uint16_t)(x01 >> 16)) & m01,
                                           e4m3x2_to_f16x2((uint16_t)(x89 & 0xFFFFu)) & m89, e4m3x2_to_f16x2((uint16_t)(x89 >> 16)) & m89};
                    mma_16816_f16(o[8 * half + 2 * w + q], x, pb[0], pb[1]);
                }
        }
    }
    template <class F> __device__ void each(int lane, F f) {
        const int gid = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int mt = 0; mt < 16; ++mt) {
            const int d = 128 * (mt >> 3) + 16 * gid + 2 * (mt & 7);
            f(2 * t4, d, o[mt][0]);
            f(2 * t4 + 1, d, o[mt][1]);
            f(2 * t4, d + 1, o[mt][2]);
            f(2 * t4 + 1, d + 1, o[mt][3]);
        }
    }
};

template <int KV, bool SCORED> struct DecodeConsumer;
template <bool SCORED> struct DecodeConsumer<KV_BF16, SCORED> { using T = DecodeBf16<SCORED>; };
template <bool SCORED> struct DecodeConsumer<KV_FP8, SCORED> { using T = DecodeE4m3<SCORED>; };

// Writes row r of a finished tile (thread's four dims d..d+3 of its
// unnormalised output, log2-unit maximum m and sum l).
template <bool SCORED>
__device__ __forceinline__ void finish_row(const PagedAttnArgs &a, const SeqSpan &q, const Tile &t, int h, int r, int d,
                                           float4 v, float m, float l, float vscale) {
    const int head = (h << a.group_shift) + (r & (a.group - 1));
    const size_t row = query_row(a, q, t, h, r);
    float lse;
    float f = row_factor(a, row, head, m, l, vscale, &lse);
    if constexpr (SCORED) {
        if ((a.first || a.last) && span_is_bad(row_span(a, q, t.t0 + (r >> a.group_shift)), row_span(a, q, t.t0),
                                               row_span(a, q, t.t0 + t.nt - 1))) {
            f = lse = __int_as_float(0x7FC00000);
            if (d == 0) atomicOr(a.seqs.err, HD_DEVERR_SPAN);
        }
    }
    uint2 w;
    w.x = pack_bf16(v.x * f, v.y * f);
    w.y = pack_bf16(v.z * f, v.w * f);
    *reinterpret_cast<uint2 *>(a.out + row * kHeadDim + d) = w;
    if (d == 0) a.lse[row] = lse;
}

template <int KV, bool SPARSE, bool SCORED>
__global__ void __launch_bounds__(kThreads, kDecodeCtasPerSm)
    paged_decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                        const __grid_constant__ PagedAttnArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr int kShift = stage_shift(KV), kKeys = 1 << kShift;
    constexpr int kHalf = kStageBytes / 2;
    float *buf = reinterpret_cast<float *>(smem + kBufOff);
    // [warps][8] maxima, [warps][8] sums, and the tile's [8] maxima and [8] sums.
    float *mx = reinterpret_cast<float *>(smem + kMlOff), *sums = mx + kWarps * kDecodeRows, *mfin = sums + kWarps * kDecodeRows;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kBarOff), *empty = full + kFulls;
    int *misc = reinterpret_cast<int *>(smem + kMiscOff), *runs = reinterpret_cast<int *>(smem + kPosOff);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const PagedSeqs &sq = a.seqs;

    if (tid == 0) {
        for (int i = 0; i < kFulls; ++i) mbar_init(&full[i], 1);
        for (int i = 0; i < kRing; ++i) mbar_init(&empty[i], team_warps(KV));
        fence_mbar_init();
    }
    __syncthreads();
    wait_for_previous_kernel();
    let_next_kernel_start();
    // This CTA's share of the call's stages.
    const int cta = blockIdx.x;
    long long x0, x1, T;
    int n, bad;
    const Start c0 = find_share(
        sq, a.num_kv_heads, cta, gridDim.x, min_units(KV),
        (SPARSE ? sq.num_tokens : sq.batch * (SCORED ? num_tiles<KV, SPARSE>(a, sq.max_tokens) : 1)) * a.num_kv_heads, kSnap, kSnap, reinterpret_cast<long long *>(buf), misc, &x0, &x1, &T, &n, &bad,
        [&](int tokens) { return num_tiles<KV, SPARSE>(a, tokens); },
        [&](const SeqSpan &q, int i) { return make_tile<KV, SPARSE, SCORED>(a, q, i).units; });
    if (bad) fill_bad_rows(a, cta, gridDim.x);
    if (x0 >= x1) return;
    // Behind the barrier a share is counted in stages done; what only cut items need waits in shared memory.
    const int share = (int)(x1 - x0);
    long long *call = reinterpret_cast<long long *>(misc + 6);   // T, x0
    if (tid == 0) {
        call[0] = T;
        call[1] = x0;
        misc[5] = n;
    }
    __syncthreads();
    Cursor c{c0.b, c0.tile, c0.h, c0.off};
    int bit;
    SeqSpan q = seq_span(sq, c.b, &bit);
    if (c.off == make_tile<KV, SPARSE, SCORED>(a, q, c.tile).units) next_item<KV, SPARSE>(a, c, q);   // a border moved to its item's end
    const int ps = 1 << sq.page_shift;
    const int box_shift = min(sq.page_shift, kShift), box_rows = 1 << box_shift;
    constexpr int kRowBytes = kHeadDim * kv_elem_bytes(KV);

    if (warp == kWarps) {
        // ---- producer ----
        const uint32_t copies = kKeys >> box_shift;   // per stage half
        int x = 0;
        int st = 0, odd = 0;   // ring slot, and kRing in the ring's odd rounds
        uint32_t ph = 0;
        bool dead = false;
        int issued = 0, copied = 0;   // stages; those whose copies were issued, the first so many
        while (x < share) {
            const Tile t = make_tile<KV, SPARSE, SCORED>(a, q, c.tile);
            const int seg = min(t.units - c.off, share - x);
            const int32_t *row = sq.table + (size_t)c.b * sq.table_stride;
            const int32_t *sel = SPARSE ? a.selected + ((size_t)(q.row0 + t.t0) * a.num_kv_heads + c.h) * a.num_selected : nullptr;
            // The segment's copies, 32 at a time: lane l looks up copy i0 + l's page and slot.
            const int first_key = (t.u0 + c.off) << kShift, total = seg * (int)copies;
            for (int i0 = 0; i0 < total; i0 += 32) {
                int page = sq.num_pages, slot = 0, pos = 0;   // page num_pages lies outside the map: the copy fills zeros
                if (i0 + lane < total) {
                    const int x_key = first_key + ((i0 + lane) << box_shift);
                    pos = key_position<SPARSE>(a, sel, t, x_key);
                    slot = x_key & (ps - 1);
                    if (pos < t.hi && pos + box_rows > t.lo) {
                        page = row[pos >> sq.page_shift];
                        if (page < 0 || page >= sq.num_pages) {
                            atomicOr(sq.err, HD_DEVERR_PAGE);
                            page = sq.num_pages;
                        }
                    }
                }
                const int cnt = min(32, total - i0);
                for (int i = 0; i < cnt; i += copies) {   // copies divides 32
                    uint8_t *dst = smem + st * kStageBytes;
                    if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(&empty[st], ph ^ 1));
                    // A barrier whose copies have not landed must not be armed again: so after a wait of its team ran out.
                    if (!dead && issued >= kFulls)
                        dead = !__all_sync(0xffffffffu, mbar_try_wait(&full[st + odd], (uint32_t)(issued / kFulls - 1) & 1));
                    const bool drop = dead || (a.drop_stage >= 0 && issued >= a.drop_stage);
                    if (!drop) {
                        ++copied;
                        const bool mine = lane >= i && lane < i + (int)copies;
                        if (SPARSE && mine) runs[st * 4 + lane - i] = pos;
                        __syncwarp();
                        if (lane == 0) mbar_arrive_expect_tx(&full[st + odd], kStageBytes);
                        __syncwarp();
                        if (mine) {
                            uint8_t *d = dst + (lane - i) * (box_rows * kRowBytes);
                            tma_load_5d(d, &kmap, &full[st + odd], 0, slot, 0, c.h, page);
                            tma_load_5d(d + kHalf, &vmap, &full[st + odd], 0, slot, 0, c.h, page);
                        }
                    }
                    ++issued;
                    if (++st == kRing) {
                        st = 0;
                        odd = kRing - odd;
                        ph ^= 1;
                    }
                }
            }
            x += seg;
            if (x < share) next_item<KV, SPARSE>(a, c, q);
        }
        // The copies land before the CTA leaves, whoever still waits for them: a lane per barrier.
        if (lane < kFulls && lane < copied && !mbar_wait(&full[lane], (uint32_t)((copied - 1 - lane) / kFulls) & 1)) dead = true;
        if (__any_sync(0xffffffffu, dead) && lane == 0) atomicOr(sq.err, HD_DEVERR_WAIT_TIMEOUT);
        return;
    }

    // ---- consumers ----
    constexpr int kTeam = team_warps(KV), kTeams = kWarps / kTeam;
    static_assert(kFulls % kTeams == 0, "a barrier serves one team");
    typename DecodeConsumer<KV, SCORED>::T cons;
    const int team = warp / kTeam;
    const int r0 = (warp % kTeam) * kWarpKeys;   // this warp's key rows of a stage
    const uint32_t base = (uint32_t)(r0 >> box_shift) * (box_rows * kRowBytes) + (r0 & (box_rows - 1)) * 128;
    const uint32_t col = box_rows * 128;
    int x = 0;
    int fb = team;             // this team's next stage: its barrier, ..
    uint32_t ph = 0;           // .. the parity of that barrier's round, ..
    int u = team;              // .. and its number from the segment's first stage
    bool dead = false;
    while (x < share) {
        const Tile t = make_tile<KV, SPARSE, SCORED>(a, q, c.tile);
        const int seg = min(t.units - c.off, share - x);
        cons.init(a, q, t, c.h, lane);
        if (warp == 0 && x + seg < share) {   // the next item's query rows into L2
            Cursor nc = c;
            SeqSpan nq = q;
            next_item<KV, SPARSE>(a, nc, nq);
            const Tile nt = make_tile<KV, SPARSE, SCORED>(a, nq, nc.tile);
            for (int i = lane; i < (nt.nt << a.group_shift) * 4; i += 32)   // 128-byte lines
                asm volatile("prefetch.global.L2 [%0];" ::"l"(a.q + query_row(a, nq, nt, nc.h, i >> 2) * kHeadDim + (i & 3) * 64));
        }
        const int pos0 = q.ctx + t.t0;
        int all_hi = pos0;                                              // every row sees up to here ..
        int all_lo = a.window ? q.ctx + t.t0 + t.nt - a.window : 0;    // .. from here
        if constexpr (SCORED) {
            all_hi = row_span(a, q, t.t0).hi;
            all_lo = row_span(a, q, t.t0 + t.nt - 1).lo;
        }
        for (; u < seg; u += kTeams) {
            const int st = fb < kRing ? fb : fb - kRing;
            if (!dead && !__all_sync(0xffffffffu, mbar_wait(&full[fb], ph))) {
                dead = true;
                if (lane == 0) atomicOr(sq.err, HD_DEVERR_WAIT_TIMEOUT);
            }
            int key0 = ((t.u0 + c.off + u) << kShift) + r0;
            if (SPARSE) key0 = runs[st * 4 + (r0 >> box_shift)] + (r0 & (box_rows - 1));
            if (!dead && key0 < t.hi && key0 + kWarpKeys > t.lo) {
                const uint8_t *stage = smem + st * kStageBytes;
                const bool whole = key0 >= all_lo && key0 + kWarpKeys - 1 <= all_hi;
                cons.consume(a, stage, stage + kHalf, base, col, key0, t.lo, t.hi, pos0, whole, lane);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
            fb += kTeams;
            if (fb >= kFulls) {
                fb -= kFulls;
                ph ^= 1;
            }
        }
        u -= seg;
        // Merge the eight warps, scaled to the rows' maxima: the upper four hand their rows to the lower four.
        const int rows = t.nt << a.group_shift;
        cons.publish(mx, sums, warp, lane);
        consumer_sync();
        auto row_max = [&](int r) {
            float m = mx[r];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) m = fmaxf(m, mx[w * kDecodeRows + r]);
            return m;
        };
        {
            const int ra = 2 * (lane & 3);
            const float wa = part_weight(mx[warp * kDecodeRows + ra], row_max(ra));
            const float wb = part_weight(mx[warp * kDecodeRows + ra + 1], row_max(ra + 1));
            if (tid < kDecodeRows) {
                const float m = row_max(tid);
                float l = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) l += sums[w * kDecodeRows + tid] * part_weight(mx[w * kDecodeRows + tid], m);
                mfin[tid] = m;
                mfin[kDecodeRows + tid] = l;
            }
            float *mine_buf = buf + (warp & (kBufs - 1)) * kBufFloats;
            if (warp >= kBufs)
                cons.each(lane, [&](int r, int d, float &v) { mine_buf[r * kRowPad + d] = v * (r & 1 ? wb : wa); });
            consumer_sync();
            if (warp < kBufs) {   // all loads, then all stores: interleaved, each would wait for the one before
                cons.each(lane, [&](int r, int d, float &v) { v = fmaf(v, r & 1 ? wb : wa, mine_buf[r * kRowPad + d]); });
                cons.each(lane, [&](int r, int d, float &v) { mine_buf[r * kRowPad + d] = v; });
            }
        }
        consumer_sync();
        const bool begins = c.off == 0, ends = c.off + seg == t.units;
        const float vscale = KV == KV_FP8 ? a.v_scale[c.h] : 1.f;
        const bool whole_item = begins && ends;
        const int slot = begins ? 2 * cta + 1 : 2 * cta;
        for (int i = tid; i < rows * (kHeadDim / 4); i += kWarps * 32) {
            const int r = i >> 6, d = (i & 63) * 4;
            float4 v = *reinterpret_cast<const float4 *>(buf + r * kRowPad + d);
#pragma unroll
            for (int k = 1; k < kBufs; ++k) {
                const float4 w = *reinterpret_cast<const float4 *>(buf + k * kBufFloats + r * kRowPad + d);
                v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
            }
            if (whole_item) {
                finish_row<SCORED>(a, q, t, c.h, r, d, v, mfin[r], mfin[kDecodeRows + r], vscale);
            } else {
                *reinterpret_cast<float4 *>(a.part_o + ((size_t)slot * kDecodeRows + r) * kHeadDim + d) = v;
                if (d == 0) a.part_ml[(size_t)slot * kDecodeRows + r] = make_float2(mfin[r], mfin[kDecodeRows + r]);
            }
        }
        if (!whole_item) {
            const long long all = call[0], item0 = call[1] + x - c.off;
            const int i0 = cta_of_unit(item0, all, misc[5]), nseg = cta_of_unit(item0 + t.units - 1, all, misc[5]) - i0 + 1;
            consumer_sync();
            if (tid == 0) {
                __threadfence();   // the block's stores (ordered by the barrier) before the ticket
                misc[4] = atomicAdd(&a.tickets[i0], 1) == nseg - 1;
                __threadfence();   // the ticket before the other pieces' loads
            }
            consumer_sync();
            if (misc[4]) {
                // A thread's four dims of a row: sixteen pieces' values and (max, sum) in flight at a time, rescaled
                // as the maximum moves -- the loads' latency, not their bytes, is what the merge waits for.
                auto piece = [&](int j) { return (size_t)(j ? 2 * (i0 + j) : 2 * i0 + 1) * kDecodeRows; };
                for (int i = tid; i < rows * (kHeadDim / 4); i += kWarps * 32) {
                    const int r = i >> 6, d = (i & 63) * 4;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    float m = -INFINITY, l = 0.f;
#pragma unroll 1
                    for (int j0 = 0; j0 < nseg; j0 += 16) {
                        float4 p[16];
                        float2 g[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const size_t at = piece(min(j0 + k, nseg - 1)) + r;
                            g[k] = __ldcg(&a.part_ml[at]);
                            p[k] = __ldcg(reinterpret_cast<const float4 *>(a.part_o + at * kHeadDim + d));
                        }
                        float top = m;
#pragma unroll
                        for (int k = 0; k < 16; ++k) top = fmaxf(top, g[k].x);
                        const float w0 = part_weight(m, top);
                        v = make_float4(v.x * w0, v.y * w0, v.z * w0, v.w * w0);
                        l *= w0;
                        m = top;
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float w = j0 + k < nseg ? part_weight(g[k].x, m) : 0.f;
                            l = fmaf(w, g[k].y, l);
                            v.x = fmaf(w, p[k].x, v.x);
                            v.y = fmaf(w, p[k].y, v.y);
                            v.z = fmaf(w, p[k].z, v.z);
                            v.w = fmaf(w, p[k].w, v.w);
                        }
                    }
                    finish_row<SCORED>(a, q, t, c.h, r, d, v, m, l, vscale);
                }
                if (tid == 0) a.tickets[i0] = 0;
            }
        }
        consumer_sync();   // the merge buffers are free again
        x += seg;
        if (x < share) next_item<KV, SPARSE>(a, c, q);
    }
}

template <int KV, bool SPARSE, bool SCORED>
cudaError_t launch(const CUtensorMap *kmap, const CUtensorMap *vmap, const PagedAttnArgs &a, int num_sms, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (!done_on_device(done, &dev)) {
        const cudaError_t e = cudaFuncSetAttribute(paged_decode_kernel<KV, SPARSE, SCORED>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        if (e != cudaSuccess) return e;
        mark_done_on_device(done, dev);
    }
    return launch_overlapping(paged_decode_kernel<KV, SPARSE, SCORED>, dim3(kDecodeCtasPerSm * num_sms), kThreads, kSmemBytes, 1, s,
                              *kmap, *vmap, a);
}

}  // namespace

cudaError_t launch_paged_decode(const CUtensorMap *kmap, const CUtensorMap *vmap, const PagedAttnArgs &a, int num_sms,
                                cudaStream_t s) {
    const bool sparse = a.selected != nullptr, scored = a.scored != 0;   // a rule and a choice of blocks do not meet
    if (a.kv_type == KV_FP8)
        return sparse   ? launch<KV_FP8, true, false>(kmap, vmap, a, num_sms, s)
               : scored ? launch<KV_FP8, false, true>(kmap, vmap, a, num_sms, s)
                        : launch<KV_FP8, false, false>(kmap, vmap, a, num_sms, s);
    return sparse   ? launch<KV_BF16, true, false>(kmap, vmap, a, num_sms, s)
           : scored ? launch<KV_BF16, false, true>(kmap, vmap, a, num_sms, s)
                    : launch<KV_BF16, false, false>(kmap, vmap, a, num_sms, s);
}

}  // namespace hd
