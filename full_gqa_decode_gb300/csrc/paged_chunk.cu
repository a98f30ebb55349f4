// Attention of chunks of new tokens over a paged cache, on the 5th-generation
// tensor cores.
//
//     S = Q K^T,  P = 2^(S log2(e)/16 - m),  O += P V
//
// with 256 query rows (heads x tokens of one kv head) and 128 keys at a time.
// A tile costs 4 x 256 x 128 x 256 flops and moves 128 KiB of K and V, so for
// long chunks the tensor cores bound it -- if the copies keep up: one SM alone
// would need 64 bytes a clock of them, all SMs together more than L2 gives.  So
// two SMs share a tile (a cluster of two CTAs, cta_group::2 MMAs): each holds
// 128 of the query rows, the scores of its rows, and half of every operand tile
// -- 64 of the 128 keys for S, 128 of the 256 dims for O -- and the pair reads
// K and V once.  Measured: 4096 tokens behind 28672 at 8 heads 687 us (1.50
// PFLOP/s, 1.5 us a tile); a prompt of 8192 at 16 heads over E4M3 pages 575 us
// (2 us a tile: the MMAs' operands, the f16 stores and the code loads all go
// through shared memory, and at 96 registers a thread the kernel keeps about
// 1.2 KB of them in local memory, which the bf16 one does not).
//
// Tensor memory (512 columns in each CTA): scores in two buffers of 128
// columns, the output of 256.  P, in 16 bits, takes the place of the scores
// that it came from and is the A operand of the second product.  The softmax of
// one tile overlaps the products of its neighbours, across items too.
//
// Roles of a CTA: eight softmax warps, two threads a row (64 scores each,
// maxima exchanged through shared memory by pairs of warps); a copy warp; the
// MMA warp (only the first CTA's issues; its barriers collect the arrivals of
// both CTAs); and stage warps, which hand a landed stage on to the MMA warp:
// with bf16 pages one warp, which only zeroes the V rows of positions that no
// row sees (they may hold NaN); with E4M3 pages four warps for K and four for V,
// which read the codes a tile ahead into registers and convert them to f16
// (exact) in the layout of the MMAs.
//
// Rows keep the reference m of their weights until a score passes it by 8 (in
// log2 units), and only then is the output in tensor memory rescaled: weights
// stay below 2^8, exact in range for bf16, and f16 weights (E4M3 pages) are
// lifted by another 2^7 away from f16's subnormals.  Sums and maxima are fp32.
// P is rounded once, to the operands' type.  In f16 (2^-11 of each weight) that
// hardly shows beside the output's rounding; in bf16 (2^-8) it adds as much as
// that does (2.4e-3 against 1.7e-3 of the output, root mean square).  The low parts
// of P through a second product, as the decode kernel takes them, would cost a
// product in two again: 4096 tokens behind 28672 905 us against 657 in the same run.
#include <climits>

#include "paged_rows.cuh"

namespace hd {
namespace {

constexpr int kTileRows = kChunkRows, kCtaRows = kTileRows / 2, kTileKeys = kChunkKeys, kKeyShift = 7;
constexpr int kSoftWarps = 8, kCopyWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1;
// Stage warps: one behind the MMA warp (bf16); two groups of four, for K and for V operands, at the next multiple of
// four warps (E4M3).  kStage: those that hand on one operand.
__host__ __device__ constexpr int first_stage_warp(int kv) { return kv == KV_FP8 ? kSoftWarps + 4 : kSoftWarps + 2; }
__host__ __device__ constexpr int stage_warps(int kv) { return kv == KV_FP8 ? 4 : 1; }
__host__ __device__ constexpr int chunk_threads(int kv) {
    return (first_stage_warp(kv) + (kv == KV_FP8 ? 2 : 1) * stage_warps(kv)) * 32;
}
// E4M3: 640 threads launch with 96 registers each; the groups of four warps then share them out by need.
// 256 x 128 + 128 x 56 + 256 x 80 <= 640 x 96.
constexpr int kSoftRegs = 128, kMiscRegs = 56, kStageRegs = 80;
static_assert(256 * kSoftRegs + 128 * kMiscRegs + 256 * kStageRegs <= 640 * 96, "a split above the launch's total never ends");
constexpr int kQBytes = kCtaRows * kHeadDim * 2;      // 64 KiB
constexpr int kSlotBytes = 32 * 1024;                 // this CTA's half of a K or V tile in 16 bits
constexpr int kSlots = 5;
constexpr int kXmOff = kQBytes + kSlots * kSlotBytes;          // [2][2][128] floats: maxima of both halves, by tile parity
constexpr int kQexpOff = kXmOff + 2 * 2 * kCtaRows * 4;   // [4][128] bytes: E4M3 pages, exponents of the rows' q
constexpr int kChunkBarOff = kQexpOff + 4 * kCtaRows;
constexpr int kChunkBars = 32;
constexpr int kChunkMiscOff = kChunkBarOff + kChunkBars * 8;
constexpr int kChunkSmem = kChunkMiscOff + 64;
constexpr int kMaxPairs = 96;
// What an item costs besides its key tiles, in tiles: its query rows and the drain of its output (about 3 us to a
// tile's 1.5).  Shares are cut by tiles plus this; short items (the first rows of a causal prompt) would otherwise
// pile up in a few shares.
constexpr int kItemCost = 2;
// Items of up to this many units are not cut: the pieces and their merge cost more than the imbalance.  Measured cut at up
// to 12 against 16: a prompt of 1500 tokens 36.5 and 30.4 us; with 0, 5 prompts of up to 4099 in 512-key windows 119 and
// 108 us.  The rows of few tokens are merged sooner: 8 sequences of 5 tokens behind 1700 24.6 and 33 us, 40 of them 50
// and 63 us; at 64 rows of 8 sequences 27 and 33 us, at 128 rows about even.
constexpr int kSnap = 16, kSnapFew = 12, kFewRows = 64;
constexpr int kMinTiles = 2 + kItemCost;              // shortest share of a pair
constexpr float kRescale = 8.f;
constexpr uint32_t kTmemCols = 512, kOutCol = 256;

// A segment -- a pair's part of an item, L key tiles -- runs in blocks of products: S(0); S(1) ; then O += P(k) V(k)
// and S(k + 2) for k = 0, 1, ..; at its end two blocks of O alone.  One commit ends a block, and block b of a segment
// is over when S(b) is complete and O holds P(b - 2) V(b - 2): it tells the softmax that its scores are there, and the
// copies which slots are free.  Blocks are counted on through the segments, L + 2 for each; segments do not overlap,
// as the next one's query rows take the place of this one's.
//
// Barriers (index into the barrier area).  A parity tells neighbouring phases apart only, so every wait is for a
// phase that the barrier cannot yet have left behind: the phase after it needs something that the waiter does next.
enum : int {
    BAR_FULL = 0,      // [5] a slot's copies have landed in this CTA (bf16 pages)
    BAR_READY = 5,     // [5] first CTA: both CTAs' halves of a slot are ready for the MMAs
    BAR_EMPTY = 10,    // [5] the MMAs that read a slot are complete (E4M3 pages)
    BAR_BLOCK = 15,    // [4] a block of products is complete, by its number modulo 4
    BAR_Q_FULL = 19,   // the query rows have landed in this CTA
    BAR_Q_READY = 20,  // first CTA: both CTAs' query rows are ready
    BAR_Q_EMPTY = 21,  // the MMAs that read the query rows are complete
    BAR_P = 22,        // [2] first CTA: the weights of both CTAs are written, by the tile's parity
    BAR_O_FULL = 24,   // a segment's output is complete
    BAR_O_FREE = 25,   // first CTA: both CTAs have read it
    BAR_DRAIN = 26,    // every MMA of the pair is complete (its only phase, at the end)
};

struct ChunkTile {
    int t0, nt, lo, hi, u0, units;   // as in the decode kernel: tokens, visible positions of any of them, key tiles
};
__device__ __forceinline__ ChunkTile make_chunk_tile(const PagedAttnArgs &a, const SeqSpan &q, int tile) {
    ChunkTile t;
    const int tt = kTileRows >> a.group_shift;
    t.t0 = tile * tt;
    t.nt = min(tt, q.n - t.t0);
    t.hi = q.ctx + t.t0 + t.nt;
    t.lo = a.window ? max(0, q.ctx + t.t0 - a.window + 1) : 0;
    t.u0 = t.lo >> kKeyShift;
    t.units = ((t.hi + kTileKeys - 1) >> kKeyShift) - t.u0;
    return t;
}
__device__ __forceinline__ int num_chunk_tiles(const PagedAttnArgs &a, int n) {
    return ((n << a.group_shift) + kTileRows - 1) / kTileRows;
}

// Units of the longest item that is not cut, by the bound on a sequence's rows of a kv head.
__device__ __forceinline__ int longest_whole(const PagedAttnArgs &a) {
    return a.seqs.max_tokens <= kFewRows >> a.group_shift ? kSnapFew : kSnap;
}

// A walk over the segments of a pair's share.
struct Segment {
    int b, tile, h;      // the item
    SeqSpan q;
    ChunkTile t;
    int u, L;            // its key tiles [u, u + L) of the item's
    int off, take, left; // units (tiles and item costs): before the segment in the item, of the segment, still to take
    int done;            // units of the share before this item's `off`

    __device__ bool settle(const PagedAttnArgs &a) {   // the next stretch that holds key tiles; false: the share is over
        for (;;) {
            take = min(t.units + kItemCost - off, left);
            u = max(off - kItemCost, 0);
            L = max(off + take - kItemCost, 0) - u;
            if (L > 0) return true;
            if (!advance(a)) return false;
        }
    }
    __device__ bool advance(const PagedAttnArgs &a) {
        left -= take;
        done += take;
        if (left <= 0) return false;
        off = 0;
        if (++h == a.num_kv_heads) {
            h = 0;
            if (++tile == num_chunk_tiles(a, q.n)) {
                tile = 0;
                int bit;
                do {
                    q = seq_span(a.seqs, ++b, &bit);
                } while (q.n == 0 && b + 1 < a.seqs.batch);
            }
            t = make_chunk_tile(a, q, tile);
        }
        return true;
    }
    __device__ bool start(const PagedAttnArgs &a, const Start &at, int share) {
        b = at.b;
        tile = at.tile;
        h = at.h;
        off = at.off;
        left = share;
        done = 0;
        int bit;
        q = seq_span(a.seqs, b, &bit);
        t = make_chunk_tile(a, q, tile);
        return settle(a);
    }
    __device__ bool next(const PagedAttnArgs &a) { return advance(a) && settle(a); }
    __device__ int key0(int k) const { return (t.u0 + u + k) << kKeyShift; }   // first position of its tile k
};

// Position in a ring of slots: index and the parity of its current round.
template <int N>
struct RingPos {
    int st = 0;
    uint32_t ph = 0;     // parity of the round that fills the slot
    bool first = true;   // whether that is the first round
    __device__ void step(int n = 1) {
        st += n;
        if (st >= N) {
            st -= N;
            ph ^= 1;
            first = false;
        }
    }
};

// ------------------------------------------------ cluster and pair-MMA PTX --
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void mbar_arrive_remote(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// The wait's other side may be the peer CTA, which releases at cluster scope; an acquire of the default scope, the
// CTA's own, would not take in what it wrote.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// Waits with the usual time limit; after one has run out (`dead`) it waits no more.
__device__ __forceinline__ void wait_thread(uint64_t *bar, uint32_t parity, bool &dead, int32_t *err) {
    if (dead || mbar_try_wait_cluster(bar, parity)) return;
    const unsigned long long t0 = globaltimer_ns();
    for (;;) {
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait_cluster(bar, parity)) return;
        if (globaltimer_ns() - t0 > kWaitLimitNs) break;
    }
    dead = true;
    atomicOr(err, HD_DEVERR_WAIT_TIMEOUT);
}
// The same for a whole warp, whose lanes go on together.
__device__ __forceinline__ void wait_warp(uint64_t *bar, uint32_t parity, bool &dead, int32_t *err) {
    wait_thread(bar, parity, dead, err);
    dead = __any_sync(0xffffffffu, dead);
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void pair_alloc(uint32_t *dst_smem) {   // whole warp, in both CTAs
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_dealloc(uint32_t taddr) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(kTmemCols) : "memory");
}
// D (+)= A B^T over both CTAs: A from shared memory (first form) or tensor memory.
__device__ __forceinline__ void pair_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
__device__ __forceinline__ void pair_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
// One arrival on the barrier at this offset in both CTAs once all MMAs issued so far are complete.
__device__ __forceinline__ void pair_commit(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
// 32 consecutive columns of this thread's lane.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Instruction descriptor for M = 256 rows of the pair: fp32 accumulator, bf16 or f16 operands, A K-major.
__host__ __device__ constexpr uint32_t pair_idesc(int n, bool bf16, int b_mn) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(kTileRows >> 4) << 24);
}

struct ChunkMaps {
    CUtensorMap q, k, v;
};

// A 16-byte load that stays in its place: eight addresses at once would not fit the stage warps' registers.
__device__ __forceinline__ uint4 load_codes(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// Four 16-byte pieces of each of four neighbouring lanes, transposed: lane q of four gets piece q of all four lanes.
__device__ __forceinline__ void transpose4(uint4 (&e)[4], int lane) {
#pragma unroll
    for (int b = 1; b <= 2; b <<= 1)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j & b) continue;
            const bool up = lane & b;
            const uint4 send = up ? e[j] : e[j | b];
            const uint4 got = make_uint4(__shfl_xor_sync(0xffffffffu, send.x, b), __shfl_xor_sync(0xffffffffu, send.y, b),
                                         __shfl_xor_sync(0xffffffffu, send.z, b), __shfl_xor_sync(0xffffffffu, send.w, b));
            if (up) e[j] = got;
            else e[j | b] = got;
        }
}

template <int KV>
__global__ void __launch_bounds__(chunk_threads(KV), 1)
    paged_chunk_kernel(const __grid_constant__ ChunkMaps maps, const __grid_constant__ PagedAttnArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr bool kFp8 = KV == KV_FP8;
    constexpr int kStage = stage_warps(KV), kStageWarp = first_stage_warp(KV);
    uint8_t *ring = smem + kQBytes;
    float *xm = reinterpret_cast<float *>(smem + kXmOff);
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + kChunkBarOff);
    int *misc = reinterpret_cast<int *>(smem + kChunkMiscOff);
    uint32_t *taddr_s = reinterpret_cast<uint32_t *>(misc + 10);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster_rank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const PagedSeqs &sq = a.seqs;
    int32_t *err = sq.err;

    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&bar[BAR_FULL + i], 1);
            mbar_init(&bar[BAR_READY + i], 2 * kStage);
            mbar_init(&bar[BAR_EMPTY + i], 1);
        }
        mbar_init(&bar[BAR_Q_FULL], 1);
        mbar_init(&bar[BAR_Q_READY], 2 * kStage);
        mbar_init(&bar[BAR_Q_EMPTY], 1);
        for (int i = 0; i < 4; ++i) mbar_init(&bar[BAR_BLOCK + i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&bar[BAR_P + i], 2 * kSoftWarps);
        mbar_init(&bar[BAR_O_FULL], 1);
        mbar_init(&bar[BAR_O_FREE], 2 * kSoftWarps);
        mbar_init(&bar[BAR_DRAIN], 1);
        fence_mbar_init();
    }
    __syncthreads();
    wait_for_previous_kernel();
    let_next_kernel_start();
    // This pair's share of the call.
    long long x0, x1, T;
    int n, bad;
    const Start c0 = find_share(
        sq, a.num_kv_heads, pair, pairs, kMinTiles, 0, longest_whole(a), INT_MAX, reinterpret_cast<long long *>(xm), misc, &x0, &x1, &T, &n, &bad,
        [&](int tokens) { return num_chunk_tiles(a, tokens); },
        [&](const SeqSpan &q, int i) { return make_chunk_tile(a, q, i).units + kItemCost; });
    if (bad) fill_bad_rows(a, blockIdx.x, gridDim.x);
    if (x0 >= x1) return;   // both CTAs of the pair
    long long *call = reinterpret_cast<long long *>(misc + 6);   // T and x0, which only cut items need again
    if (tid == 0) {
        call[0] = T;
        call[1] = x0;
        misc[5] = n;
    }
    if (warp == kMmaWarp) pair_alloc(taddr_s);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();   // the peer's barriers are initialised
    tc_fence_after();
    const uint32_t tmem = *taddr_s;
    const int share = (int)(x1 - x0);
    Segment w;
    bool more = w.start(a, c0, share);   // no role has work when the share holds item costs alone
    bool dead = false;
    const int ps = 1 << sq.page_shift;
    // Whole-warp wait for the end of block i.
    auto wait_block = [&](int i) { wait_warp(&bar[BAR_BLOCK + (i & 3)], (uint32_t)(i >> 2) & 1, dead, err); };
    // Pages of a tile's eight groups of 16 keys, one per lane; a page that no row sees lies outside the map.
    auto pages_of = [&](const Segment &x, int k) {
        const int pos = x.key0(k) + 16 * (lane & 7), first = pos & ~(ps - 1);
        int page = sq.num_pages;
        if (first < x.t.hi && first + ps > x.t.lo) {
            page = sq.table[(size_t)x.b * sq.table_stride + (pos >> sq.page_shift)];
            if (page < 0 || page >= sq.num_pages) {
                atomicOr(err, HD_DEVERR_PAGE);
                page = sq.num_pages;
            }
        }
        return page;
    };

    // E4M3: each group of four warps takes its registers on entry to its role.
    if (warp >= kSoftWarps && warp < kStageWarp) {
    if (kFp8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMiscRegs));

    if (warp == kCopyWarp) {
        // ---- copies: a segment's query rows, then K(0), K(1), V(0), K(2), V(1), .., V(L - 1) (E4M3 pages: the stage
        // warps read those) ----
        const int rk_shift = min(sq.page_shift, 6), rv_shift = min(sq.page_shift, 7);
        // bf16 pages of fewer than 64 slots: a K copy per column group, so that the 64 keys' rows of a group lie
        // together as the MMA wants them.
        const bool split = rk_shift < 6;
        const int tok = kCtaRows >> a.group_shift;
        RingPos<kSlots> pos;
        int issued = 0, blocks = 0;   // blocks: before this segment
        int copied = 0;               // operands whose copies were issued: the first so many
        uint32_t q_copied = 0;        // segments whose query rows were
        int last_read = -1;
        for (uint32_t seg = 0; more; ++seg) {
            int pg = kFp8 ? 0 : pages_of(w, 0), pg_v = 0;
            if (seg) {
                wait_warp(&bar[BAR_Q_EMPTY], (seg - 1) & 1, dead, err);
                // A barrier whose copy has not landed must not be armed again: so after a wait of others ran out.
                dead = __any_sync(0xffffffffu, dead || !mbar_try_wait(&bar[BAR_Q_FULL], (seg - 1) & 1));
            }
            if (!dead) ++q_copied;
            if (lane == 0 && !dead) {
                mbar_arrive_expect_tx(&bar[BAR_Q_FULL], kQBytes);
                tma_load_4d(smem, &maps.q, &bar[BAR_Q_FULL], 0, w.h << a.group_shift, w.q.row0 + w.t.t0 + rank * tok, 0);
            }
            for (int i = 0; !kFp8 && i <= w.L; ++i) {
                const int pg_next = i + 1 < w.L ? pages_of(w, i + 1) : 0;
#pragma unroll
                for (int kind = 0; kind < 2; ++kind) {   // K(i), then V(i - 1)
                    if (kind == 0 ? i >= w.L : i == 0) continue;
                    // The operand is read by block r, the slot's last one by the block in lane `slot` of last_read.  A
                    // barrier of four phases tells the end of block r - 4 or later, as block r does not end without
                    // this copy.
                    const int r = blocks + (kind == 0 ? i : i + 1);
                    const int before = max(__shfl_sync(0xffffffffu, last_read, pos.st), r - 4);
                    if (before >= 0) wait_block(before);
                    if (lane == pos.st) last_read = r;
                    uint8_t *dst = ring + pos.st * kSlotBytes;
                    uint64_t *full = &bar[BAR_FULL + pos.st];
                    if (!pos.first) dead = __any_sync(0xffffffffu, dead || !mbar_try_wait(full, pos.ph ^ 1));
                    const bool drop = dead || (a.drop_stage >= 0 && issued >= a.drop_stage);
                    if (!drop) ++copied;
                    if (!drop && lane == 0) mbar_arrive_expect_tx(full, kSlotBytes);
                    __syncwarp();
                    const int shift = kind == 0 ? rk_shift : rv_shift;
                    const int run = kind == 0 && split ? lane >> 2 : lane;
                    const int col = kind == 0 ? (split ? lane & 3 : 0) : 2 * rank;
                    const int total = kind == 0 ? (64 >> rk_shift) * (split ? 4 : 1) : 128 >> rv_shift;
                    const uint32_t off = kind == 0 ? (split ? col * 8192 + (run << shift) * 128 : 0) : (run << shift) * 256;
                    const int first = (kind == 0 ? 64 * rank : 0) + (run << shift);   // of this copy's keys in the tile
                    const int page = __shfl_sync(0xffffffffu, kind == 0 ? pg : pg_v, (first >> 4) & 7);
                    if (!drop && lane < total) {
                        const int slot = (w.key0(kind == 0 ? i : i - 1) + first) & (ps - 1);
                        tma_load_5d(dst + off, kind == 0 ? &maps.k : &maps.v, full, 0, slot, col, w.h, page);
                    }
                    ++issued;
                    pos.step();
                }
                pg_v = pg;
                pg = pg_next;
            }
            blocks += w.L + 2;
            more = w.next(a);
            if (more && lane == 0)   // the next segment's query rows into L2
                asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                                 reinterpret_cast<uint64_t>(&maps.q)),
                             "r"(0), "r"(w.h << a.group_shift), "r"(w.q.row0 + w.t.t0 + rank * tok), "r"(0)
                             : "memory");
        }
        // This CTA's copies land before it leaves, whoever still waits for them: a lane per slot, and one for the rows.
        bool landed = true;
        if (lane < kSlots && lane < copied) landed = mbar_wait(&bar[BAR_FULL + lane], (uint32_t)((copied - 1 - lane) / kSlots) & 1);
        if (lane == kSlots && q_copied) landed = mbar_wait(&bar[BAR_Q_FULL], (q_copied - 1) & 1);
        if (!landed) atomicOr(err, HD_DEVERR_WAIT_TIMEOUT);
    } else if (warp == kMmaWarp) {
        // ---- products, block by block; once a wait has run out the commits go on alone, for those who wait for them ----
        if (rank == 0 && lane == 0) {
            constexpr uint32_t kIdS = pair_idesc(128, !kFp8, 0), kIdO = pair_idesc(256, !kFp8, 1);
            const int rv_shift = kFp8 ? 7 : min(sq.page_shift, 7);
            const uint64_t qd0 = umma_desc(smem_u32(smem), 16, 1024, 2);
            const uint64_t kd0 = umma_desc(smem_u32(ring), 16, 1024, 2);
            const uint64_t vd0 = umma_desc(smem_u32(ring), 128u << rv_shift, 1024, 2);
            uint32_t v_step[8];   // offsets of a V slot's 16-key steps
#pragma unroll
            for (int t = 0; t < 8; ++t)
                v_step[t] = (((uint32_t)(16 * t) >> rv_shift << rv_shift) * 256 + ((uint32_t)(16 * t) & ((1u << rv_shift) - 1)) * 128) >> 4;
            RingPos<kSlots> pos;
            int blocks = 0, tiles = 0;   // before this segment
            for (uint32_t seg = 0; more; ++seg) {
                for (int i = 0; i < w.L + 2; ++i) {
                    if (i >= 2) {
                        const int g = tiles + i - 2;
                        if (i == 2 && seg) wait_thread(&bar[BAR_O_FREE], (seg - 1) & 1, dead, err);
                        wait_thread(&bar[BAR_READY + pos.st], pos.ph, dead, err);
                        wait_thread(&bar[BAR_P + (g & 1)], (uint32_t)(g >> 1) & 1, dead, err);
                        tc_fence_after();
                        const uint64_t vd = vd0 + (uint64_t)((uint32_t)pos.st * kSlotBytes >> 4);
                        const uint32_t p = tmem + (uint32_t)(g & 1) * 128;
                        if (!dead) {
#pragma unroll
                            for (int t = 0; t < 8; ++t)
                                pair_mma_ts(tmem + kOutCol, p + 8 * t, vd + v_step[t], kIdO, i > 2 || t > 0);
                        }
                        if (kFp8) pair_commit(&bar[BAR_EMPTY + pos.st]);
                        pos.step();
                    }
                    if (i < w.L) {
                        if (i == 0) wait_thread(&bar[BAR_Q_READY], seg & 1, dead, err);
                        wait_thread(&bar[BAR_READY + pos.st], pos.ph, dead, err);
                        tc_fence_after();
                        const uint64_t kd = kd0 + (uint64_t)((uint32_t)pos.st * kSlotBytes >> 4);
                        const uint32_t d = tmem + (uint32_t)((tiles + i) & 1) * 128;
                        if (!dead) {
#pragma unroll
                            for (int kk = 0; kk < 16; ++kk)
                                pair_mma_ss(d, qd0 + (uint64_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                                            kd + (uint64_t)(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), kIdS, kk > 0);
                        }
                        if (kFp8) pair_commit(&bar[BAR_EMPTY + pos.st]);
                        pos.step();
                    }
                    pair_commit(&bar[BAR_BLOCK + ((blocks + i) & 3)]);
                    if (i == w.L - 1) pair_commit(&bar[BAR_Q_EMPTY]);
                    if (i == w.L + 1) pair_commit(&bar[BAR_O_FULL]);
                }
                blocks += w.L + 2;
                tiles += w.L;
                more = w.next(a);
            }
            pair_commit(&bar[BAR_DRAIN]);
        }
    }
    } else if (kFp8 && warp >= kStageWarp) {
        // ---- E4M3 operands ----
        if (kFp8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kStageRegs));
        // The codes of the next operand wait in registers, eight 16-byte chunks a thread.  A warp's lanes take two (K)
        // or four (V) whole rows at a time, in an order that makes both the reads whole lines and the f16 stores free
        // of bank conflicts: of eight lanes, four take neighbouring chunks of a row and four those of the row beside it.
        const int sw = (warp - kStageWarp) & 3, row2 = (lane >> 2) & 1;
        const uint32_t ready0 = dsmem_addr(&bar[BAR_READY], 0);
        uint4 codes[8];
        auto put = [&](uint8_t *slot, const uint4 &x, int row, int c, uint32_t col) {
            const uint32_t cw[4] = {x.x, x.y, x.z, x.w};
            uint32_t f[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[2 * j] = e4m3x2_to_f16x2((uint16_t)(cw[j] & 0xFFFFu));
                f[2 * j + 1] = e4m3x2_to_f16x2((uint16_t)(cw[j] >> 16));
            }
            uint8_t *dst = slot + (uint32_t)(c >> 2) * col + (uint32_t)row * 128;
            *reinterpret_cast<uint4 *>(dst + (((2 * (c & 3)) ^ (row & 7)) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<uint4 *>(dst + (((2 * (c & 3) + 1) ^ (row & 7)) << 4)) = make_uint4(f[4], f[5], f[6], f[7]);
        };
        RingPos<kSlots> pos;
        auto wait_slot = [&]() {
            if (!pos.first) wait_warp(&bar[BAR_EMPTY + pos.st], pos.ph ^ 1, dead, err);
        };
        int number = 0;   // of the operand at pos, as the copy warp counts them
        auto to_operand = [&](int n) {
            pos.step(n);
            number += n;
        };
        auto hand_on = [&]() {
            fence_async_smem();
            __syncwarp();
            const bool drop = a.drop_stage >= 0 && number >= a.drop_stage;
            if (lane == 0 && !drop) mbar_arrive_remote(ready0 + 8 * pos.st);
        };
        if (warp < kStageWarp + 4) {
            // K(k), of a segment's loads the first and then number 2 k - 1: this CTA's 64 keys x 16 chunks.
            const uint32_t q_ready = dsmem_addr(&bar[BAR_Q_READY], 0);
            const int chunk = (lane & 3) | (lane >> 3 << 2);
            auto load = [&](int k) {
                const int pg = pages_of(w, k), key0 = w.key0(k);
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    const int key = 64 * rank + s * 8 + sw * 2 + row2, page = __shfl_sync(0xffffffffu, pg, key >> 4);
                    const size_t at = (size_t)page * a.page_stride +
                                      (((size_t)w.h << sq.page_shift) + ((key0 + key) & (ps - 1))) * kHeadDim + 16 * chunk;
                    codes[s] = page < sq.num_pages ? load_codes(a.k_codes + at) : make_uint4(0u, 0u, 0u, 0u);
                }
            };
            if (more) load(0);
            for (uint32_t seg = 0; more; ++seg) {
                {
                    // A thread's row of q in f16, scaled by the power of two that brings its largest value below 2
                    // (and by the sign of the K scale); the softmax multiplies the scores back.
                    wait_warp(&bar[BAR_Q_FULL], seg & 1, dead, err);
                    const int row = sw * 32 + lane;
                    uint8_t *qrow = smem + row * 128;
                    uint32_t top = 0;
#pragma unroll 8
                    for (int c = 0; c < 32; ++c) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(qrow + (c >> 3) * 16384 + (((c & 7) ^ (row & 7)) << 4));
                        const uint32_t cw[4] = {x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu, x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu};
#pragma unroll
                        for (int j = 0; j < 4; ++j) top = max(top, max(cw[j] & 0xFFFFu, cw[j] >> 16));
                    }
                    const int ex = min(max((int)(top >> 7), 1), 253);
                    const float down = copysignf(__uint_as_float((uint32_t)(254 - ex) << 23), a.k_scale[w.h]);
#pragma unroll 8
                    for (int c = 0; c < 32; ++c) {
                        uint4 *at = reinterpret_cast<uint4 *>(qrow + (c >> 3) * 16384 + (((c & 7) ^ (row & 7)) << 4));
                        uint4 x = *at;
                        auto half2 = [&](uint32_t v) {
                            return pack_f16(__uint_as_float(v << 16) * down, __uint_as_float(v & 0xFFFF0000u) * down);
                        };
                        *at = make_uint4(half2(x.x), half2(x.y), half2(x.z), half2(x.w));
                    }
                    smem[kQexpOff + (seg & 3) * kCtaRows + row] = (uint8_t)ex;
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote(q_ready);
                }
                const int L = w.L;
                for (int k = 0; k < L; ++k) {
                    wait_slot();
                    uint8_t *slot = ring + pos.st * kSlotBytes;
#pragma unroll
                    for (int s = 0; s < 8; ++s) put(slot, codes[s], s * 8 + sw * 2 + row2, chunk, 8192);
                    hand_on();
                    to_operand(k + 1 < L ? (k ? 2 : 1) : (k ? 3 : 2));   // to the next K, over the last V's at the end
                    if (k + 1 < L) load(k + 1);
                }
                more = w.next(a);
                if (more) load(0);
            }
        } else {
            // V(k), of a segment's loads number 2 k + 2 and the last: 128 keys x 8 chunks of this CTA's dims.  Rows of
            // positions that no query row sees are zero, whatever their slots hold.
            const int chunk = (lane & 3) | (lane >> 3 & 1) << 2, row4 = row2 + 2 * (lane >> 4);
            auto load = [&](int k) {
                const int pg = pages_of(w, k), key0 = w.key0(k);
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    const int key = s * 16 + sw * 4 + row4, page = __shfl_sync(0xffffffffu, pg, key >> 4), p = key0 + key;
                    const size_t at = (size_t)page * a.page_stride +
                                      (((size_t)w.h << sq.page_shift) + (p & (ps - 1))) * kHeadDim + 128 * rank + 16 * chunk;
                    codes[s] = page < sq.num_pages && p >= w.t.lo && p < w.t.hi ? load_codes(a.v_codes + at)
                                                                               : make_uint4(0u, 0u, 0u, 0u);
                }
            };
            if (more) load(0);
            while (more) {
                const int L = w.L;
                to_operand(L > 1 ? 2 : 1);
                for (int k = 0; k < L; ++k) {
                    wait_slot();
                    uint8_t *slot = ring + pos.st * kSlotBytes;
#pragma unroll
                    for (int s = 0; s < 8; ++s) put(slot, codes[s], s * 16 + sw * 4 + row4, chunk, 16384);
                    hand_on();
                    to_operand(k + 2 < L ? 2 : 1);
                    if (k + 1 < L) load(k + 1);
                }
                more = w.next(a);
                if (more) load(0);
            }
        }
    } else if (!kFp8 && warp == kStageWarp) {
        // ---- bf16 stages: hand what has landed on to the MMAs ----
        const uint32_t ready0 = dsmem_addr(&bar[BAR_READY], 0), q_ready = dsmem_addr(&bar[BAR_Q_READY], 0);
        const int rv_shift = min(sq.page_shift, 7);
        RingPos<kSlots> pos;
        for (uint32_t seg = 0; more; ++seg) {
            wait_warp(&bar[BAR_Q_FULL], seg & 1, dead, err);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(q_ready);
            for (int i = 0; i <= w.L; ++i) {
#pragma unroll
                for (int kind = 0; kind < 2; ++kind) {   // K(i), then V(i - 1)
                    if (kind == 0 ? i >= w.L : i == 0) continue;
                    uint8_t *slot = ring + pos.st * kSlotBytes;
                    wait_warp(&bar[BAR_FULL + pos.st], pos.ph, dead, err);
                    const int key0 = w.key0(i - 1);
                    if (kind == 1 && (key0 < w.t.lo || key0 + kTileKeys > w.t.hi)) {
                        // Rows of positions that no query row sees: zero, whatever their slots hold.
                        for (int r = 0; r < kTileKeys; ++r) {
                            if (key0 + r >= w.t.lo && key0 + r < w.t.hi) continue;
                            const uint32_t at = (uint32_t)(r >> rv_shift << rv_shift) * 256 +
                                                (uint32_t)(r & ((1 << rv_shift) - 1)) * 128 +
                                                (lane >> 3 & 1) * (128u << rv_shift) + (lane & 7) * 16;
                            if (lane < 16) *reinterpret_cast<uint4 *>(slot + at) = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote(ready0 + 8 * pos.st);
                    pos.step();
                }
            }
            more = w.next(a);
        }
    } else if (warp < kSoftWarps) {
        // ---- softmax: thread (row, half of the tile's keys) ----
        if (kFp8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int half = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);   // lane 32 (warp % 4) in the upper half-word
        const uint32_t p_bar = dsmem_addr(&bar[BAR_P], 0), o_free = dsmem_addr(&bar[BAR_O_FREE], 0);
        auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 3)) : "memory"); };
        auto soft_sync = [&]() { asm volatile("bar.sync 5, 256;" ::: "memory"); };
        const float lift = kFp8 ? 7.f : 0.f;
        int blocks = 0, tiles = 0;   // before this segment
        for (uint32_t seg = 0; more; ++seg) {
        float m = -INFINITY, l = 0.f, scale = kQScale;
        const int r = rank * kCtaRows + row;
        const int hi_pos = w.q.ctx + w.t.t0 + (r >> a.group_shift), lo_pos = a.window ? hi_pos - a.window + 1 : 0;
        const int all_hi = w.q.ctx + w.t.t0;                                            // every row sees up to here ..
        const int all_lo = a.window ? w.q.ctx + w.t.t0 + w.t.nt - a.window : 0;        // .. from here
        const int rows_here = (w.t.nt << a.group_shift) - rank * kCtaRows;              // valid rows of this CTA
        const bool idle = (warp & 3) * 32 >= rows_here;                                  // none of this warp's rows exists
        for (int k = 0; k < w.L; ++k) {
            const int g = tiles + k;
            const uint32_t buf = lanes + (uint32_t)(g & 1) * 128;
            wait_block(blocks + k);
            if (kFp8 && k == 0) {
                const uint32_t ex = smem[kQexpOff + (seg & 3) * kCtaRows + row];
                scale = fmaxf(__uint_as_float(ex << 23) * fabsf(a.k_scale[w.h] * kQScale), 1e-37f);
            }
            if (!idle) {
                tc_fence_after();
                float s[64];
                tmem_ld32(buf + half * 64, *reinterpret_cast<float(*)[32]>(s));
                tmem_ld32(buf + half * 64 + 32, *reinterpret_cast<float(*)[32]>(s + 32));
                const int key0 = w.key0(k) + half * 64;
                if (key0 < all_lo || key0 + 63 > all_hi) {
                    const int from = lo_pos - key0, to = hi_pos - key0;
#pragma unroll
                    for (int i = 0; i < 64; ++i) s[i] = i >= from && i <= to ? s[i] : -INFINITY;
                }
                float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int i = 4; i < 64; ++i) mx[i & 3] = fmaxf(mx[i & 3], s[i]);
                float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                float *x = xm + (g & 1) * 2 * kCtaRows;
                x[half * kCtaRows + row] = top;
                pair_sync();
                top = fmaxf(top, x[(half ^ 1) * kCtaRows + row]);
                top *= scale;
                float alpha = 1.f;
                if (top > m + kRescale) {   // also a row's first key: m = -inf
                    alpha = fast_exp2(m - top);   // m = -inf: 0
                    m = top;
                    l *= alpha;
                }
                if (k > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                    wait_block(blocks + k + 1);   // O holds tile k - 1
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 128; c += 32) {
                        float o[32];
                        uint32_t ow[32];
                        tmem_ld32(lanes + kOutCol + half * 128 + c, o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) ow[i] = __float_as_uint(o[i] * alpha);
                        tmem_st32(lanes + kOutCol + half * 128 + c, ow);
                    }
                }
                const float ref = m == -INFINITY ? 0.f : m - lift;
                uint32_t pw[32];
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float p0 = fast_exp2(fmaf(s[2 * i], scale, -ref)), p1 = fast_exp2(fmaf(s[2 * i + 1], scale, -ref));
                    sum[i & 1] += p0;
                    sum[2 + (i & 1)] += p1;
                    pw[i] = kFp8 ? pack_f16(p0, p1) : pack_bf16(p0, p1);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tmem_st32(buf + half * 32, pw);
                tmem_wait_st();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(p_bar + 8 * (uint32_t)(g & 1));

        }
            // ---- the segment's output ----
            {
                float *x = xm + ((tiles + w.L) & 1) * 2 * kCtaRows;
                if (!idle) {
                    x[half * kCtaRows + row] = l;
                    pair_sync();
                    l += x[(half ^ 1) * kCtaRows + row];
                    pair_sync();
                }
                const bool whole = w.L == w.t.units, live = row < rows_here;
                const float ml_m = m - lift;
                const int slot = w.u == 0 ? 2 * pair + 1 : 2 * pair;
                const size_t prow = (size_t)slot * kTileRows + r;
                const float vscale = kFp8 ? a.v_scale[w.h] : 1.f;
                const int head = (w.h << a.group_shift) + (r & (a.group - 1));
                const size_t orow = (size_t)(w.q.row0 + w.t.t0 + (r >> a.group_shift)) * a.num_q_heads + head;
                float f = 1.f;
                if (live) {
                    if (whole) {
                        float lse;
                        f = row_factor(a, orow, head, ml_m, l, vscale, &lse);
                        if (half == 0) a.lse[orow] = lse;
                    } else if (half == 0) {
                        a.part_ml[prow] = make_float2(ml_m, l);
                    }
                }
                wait_warp(&bar[BAR_O_FULL], seg & 1, dead, err);
                tc_fence_after();
                if (!idle) {
                    // A lane holds a row; four lanes trade pieces so that each store writes 64 bytes of a row together
                    // (a row a lane, 16 bytes at a time, took 4 us an item).
                    const int r4 = row & ~3, piece = lane & 3;
                    size_t row4[4];
                    bool live4[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        live4[j] = r4 + j < rows_here;
                        const int rr = rank * kCtaRows + r4 + j;
                        row4[j] = whole ? (size_t)(w.q.row0 + w.t.t0 + (rr >> a.group_shift)) * a.num_q_heads +
                                              (w.h << a.group_shift) + (rr & (a.group - 1))
                                        : (size_t)slot * kTileRows + rr;
                    }
#pragma unroll 1
                    for (int c = half * 128; c < half * 128 + 128; c += 32) {
                        float o[32];
                        tmem_ld32(lanes + kOutCol + c, o);
                        uint4 e[4];
                        if (whole) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                e[i] = make_uint4(pack_bf16(o[8 * i] * f, o[8 * i + 1] * f), pack_bf16(o[8 * i + 2] * f, o[8 * i + 3] * f),
                                                  pack_bf16(o[8 * i + 4] * f, o[8 * i + 5] * f), pack_bf16(o[8 * i + 6] * f, o[8 * i + 7] * f));
                            transpose4(e, lane);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (live4[j]) *reinterpret_cast<uint4 *>(a.out + row4[j] * kHeadDim + c + 8 * piece) = e[j];
                        } else {
#pragma unroll
                            for (int p = 0; p < 2; ++p) {
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    e[i] = make_uint4(__float_as_uint(o[16 * p + 4 * i]), __float_as_uint(o[16 * p + 4 * i + 1]),
                                                      __float_as_uint(o[16 * p + 4 * i + 2]), __float_as_uint(o[16 * p + 4 * i + 3]));
                                transpose4(e, lane);
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    if (live4[j])
                                        *reinterpret_cast<uint4 *>(a.part_o + row4[j] * kHeadDim + c + 16 * p + 4 * piece) = e[j];
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(o_free);
                if (!whole) {
                    // The last of the item's pieces to arrive (for this CTA's rows) merges them.
                    const long long all = call[0], from = call[1] + w.done - w.off + kItemCost;   // the item's first tile
                    const int i0 = cta_of_unit(from, all, misc[5]), nseg = cta_of_unit(from + w.t.units - 1, all, misc[5]) - i0 + 1;
                    soft_sync();
                    if (tid == 0) {
                        __threadfence();   // the block's stores (ordered by the barrier) before the ticket
                        misc[4] = atomicAdd(&a.tickets[2 * i0 + rank], 1) == nseg - 1;
                        __threadfence();   // the ticket before the other pieces' loads
                    }
                    soft_sync();
                    if (misc[4]) {
                        // First each row's maximum and factor, by a thread a row; then the outputs, a thread's four dims of
                        // kMergeRows rows and two pieces at a time in flight.
                        const int d = (tid & 63) * 4, rows = min(rows_here, kCtaRows);
                        auto piece = [&](int j) { return (size_t)(j ? 2 * (i0 + j) : 2 * i0 + 1) * kTileRows + rank * kCtaRows; };
                        auto out_row = [&](int rr) {
                            const int rt = rank * kCtaRows + rr;
                            return (size_t)(w.q.row0 + w.t.t0 + (rt >> a.group_shift)) * a.num_q_heads +
                                   (w.h << a.group_shift) + (rt & (a.group - 1));
                        };
                        if (half == 0 && live) {
                            float mm = -INFINITY, ll = 0.f;
#pragma unroll 2
                            for (int j = 0; j < nseg; ++j) {
                                const float2 ml = __ldcg(&a.part_ml[piece(j) + row]);
                                const float top = fmaxf(mm, ml.x);
                                ll = ll * part_weight(mm, top) + ml.y * part_weight(ml.x, top);
                                mm = top;
                            }
                            float lse;
                            xm[kCtaRows + row] = row_factor(a, orow, head, mm, ll, vscale, &lse);
                            xm[row] = mm;
                            a.lse[orow] = lse;
                        }
                        soft_sync();
                        constexpr int kMergeRows = kFp8 ? 4 : 8;
#pragma unroll 1
                        for (int r0 = tid >> 6; r0 < rows; r0 += 4 * kMergeRows) {
                            float4 v[kMergeRows];
#pragma unroll
                            for (int i = 0; i < kMergeRows; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
                            for (int j0 = 0; j0 < nseg; j0 += 2) {
                                float4 p[kMergeRows][2];
                                float pm[kMergeRows][2];
#pragma unroll
                                for (int i = 0; i < kMergeRows; ++i)
#pragma unroll
                                    for (int k = 0; k < 2; ++k) {
                                        const size_t at = piece(min(j0 + k, nseg - 1)) + min(r0 + 4 * i, rows - 1);
                                        pm[i][k] = __ldcg(&a.part_ml[at].x);
                                        p[i][k] = __ldcg(reinterpret_cast<const float4 *>(a.part_o + at * kHeadDim + d));
                                    }
#pragma unroll
                                for (int i = 0; i < kMergeRows; ++i) {
                                    const float top = xm[min(r0 + 4 * i, rows - 1)];
                                    const float wa = part_weight(pm[i][0], top);
                                    const float wb = j0 + 1 < nseg ? part_weight(pm[i][1], top) : 0.f;
                                    v[i].x += wa * p[i][0].x + wb * p[i][1].x;
                                    v[i].y += wa * p[i][0].y + wb * p[i][1].y;
                                    v[i].z += wa * p[i][0].z + wb * p[i][1].z;
                                    v[i].w += wa * p[i][0].w + wb * p[i][1].w;
                                }
                            }
#pragma unroll
                            for (int i = 0; i < kMergeRows; ++i) {
                                const int rr = r0 + 4 * i;
                                if (rr >= rows) break;
                                const float ff = xm[kCtaRows + rr];
                                *reinterpret_cast<uint2 *>(a.out + out_row(rr) * kHeadDim + d) =
                                    make_uint2(pack_bf16(v[i].x * ff, v[i].y * ff), pack_bf16(v[i].z * ff, v[i].w * ff));
                            }
                        }
                        if (tid == 0) a.tickets[2 * i0 + rank] = 0;
                    }
                    soft_sync();
                }
            }
            blocks += w.L + 2;
            tiles += w.L;
            more = w.next(a);
        }
    }
    __syncwarp();
    // No CTA leaves, and no tensor memory is freed, while MMAs of the pair or its peer's arrivals may still reach it: when
    // waits have run out, nobody else has waited for the last ones.
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (warp == kMmaWarp) {
        if (!__all_sync(0xffffffffu, mbar_wait(&bar[BAR_DRAIN], 0)) && lane == 0) atomicOr(err, HD_DEVERR_WAIT_TIMEOUT);
        tc_fence_after();
        pair_dealloc(tmem);
    }
}

template <int KV>
cudaError_t chunk_setup(int *pairs) {
    static std::atomic<uint64_t> done{0};
    static std::atomic<int> limit[64];
    int dev = 0;
    if (!done_on_device(done, &dev)) {
        cudaError_t e = cudaFuncSetAttribute(paged_chunk_kernel<KV>, cudaFuncAttributeMaxDynamicSharedMemorySize, kChunkSmem);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg{};
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim = {2, 1, 1};
        cfg.gridDim = dim3(2 * kMaxPairs);
        cfg.blockDim = dim3(chunk_threads(KV));
        cfg.dynamicSmemBytes = kChunkSmem;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, paged_chunk_kernel<KV>, &cfg);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) limit[dev].store(n, std::memory_order_relaxed);
        *pairs = n;
        mark_done_on_device(done, dev);
        return cudaSuccess;
    }
    *pairs = limit[dev].load(std::memory_order_relaxed);
    return cudaSuccess;
}

template <int KV>
cudaError_t launch_chunk(const ChunkMaps &maps, const PagedAttnArgs &a, cudaStream_t s) {
    int pairs = 0;
    cudaError_t e = chunk_setup<KV>(&pairs);
    if (e != cudaSuccess) return e;
    if (pairs > kMaxPairs) pairs = kMaxPairs;
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    return launch_overlapping(paged_chunk_kernel<KV>, dim3(2 * pairs), chunk_threads(KV), kChunkSmem, 2, s, maps, a);
}

}  // namespace

cudaError_t launch_paged_chunk(const CUtensorMap *qmap, const CUtensorMap *kmap, const CUtensorMap *vmap,
                               const PagedAttnArgs &a, cudaStream_t s) {
    ChunkMaps maps{*qmap, *kmap, *vmap};
    return a.kv_type == KV_FP8 ? launch_chunk<KV_FP8>(maps, a, s) : launch_chunk<KV_BF16>(maps, a, s);
}

}  // namespace hd
