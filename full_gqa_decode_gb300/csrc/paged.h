// Internal declarations of the paged-cache operators: kernel arguments and
// launchers.  Not part of the C ABI.
#pragma once

#include "hd_internal.h"

namespace hd {

constexpr int kMinPageShift = 4;    // pages of 16 ..
constexpr int kMaxPageShift = 8;    // .. 256 slots, a power of two
constexpr int kDecodeRows = 8;      // query rows per kv head (heads x tokens) of one decode tile
constexpr int kDecodeCtasPerSm = 1;
constexpr int kChunkRows = 256;     // query rows of one chunk tile (a pair of CTAs)
constexpr int kChunkKeys = 128;     // keys of one chunk tile
constexpr int kPagedTickets = 1024;  // at least the CTAs of a paged attention grid
constexpr int kMaxSelectBlocks = 16384;   // blocks of one sequence that select_pages ranks (192 KiB of keys)

// The sequences of a paged call.  A sequence's new tokens are rows
// [offsets[b], offsets[b + 1]) of q / k / v / out (offsets null: row b); they
// sit at positions context[b] + t.
struct PagedSeqs {
    const int32_t *table;      // [batch][table_stride]: page of block i
    int64_t table_stride;
    const int32_t *context;    // [batch]
    const int32_t *offsets;    // [batch + 1] or null
    int32_t batch, num_tokens, max_tokens, max_blocks;
    int32_t max_context;       // bound of this call on context[b]
    int32_t max_position;      // last position with a rotary table row
    int32_t page_shift, num_pages;
    int32_t *err;
};

struct PagedAppendArgs {
    PagedSeqs seqs;
    const __nv_bfloat16 *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;   // elements between rows
    __nv_bfloat16 *q_rot;                   // [num_tokens][Hq][D] or null
    void *cache_k, *cache_v;
    int64_t page_stride;                    // elements
    const float *k_scale, *v_scale;         // E4M3 or null
    __nv_bfloat16 *bounds;                  // [num_pages][Hkv][2][D] or null
    const float2 *rope;                     // [max_position + 1][rotary_dim / 2]
    int32_t rotary_dim, num_q_heads, num_kv_heads, kv_type;
};

// Attention over pages: dense (every visible position) or over selected
// blocks (`selected`: [num_tokens][Hkv][num_selected] ascending block numbers,
// -1 past the end).
struct PagedAttnArgs {
    PagedSeqs seqs;
    const __nv_bfloat16 *q;    // rotated [num_tokens][Hq][D]
    const int32_t *selected;
    int32_t num_selected;
    const uint8_t *k_codes, *v_codes;   // E4M3 pages (the chunk kernel reads them without a tensor map)
    int64_t page_stride;                // elements
    const float *k_scale, *v_scale;
    const float *sink, *gate;
    __nv_bfloat16 *out;
    float *lse;
    float *part_o;             // partial rows of cut items, two slots per CTA
    float2 *part_ml;           // (max in log2 units, sum)
    int32_t *tickets;          // [CTAs], zero between calls
    int32_t num_q_heads, num_kv_heads, group, group_shift;   // group: 1, 2, 4 or 8 = 1 << group_shift
    int32_t window;            // sliding layers; 0: all positions
    int32_t kv_type;
    int32_t drop_stage;        // test hook: the producers stop issuing at this stage (-1: off)
};

struct PagedSelectArgs {
    PagedSeqs seqs;
    const __nv_bfloat16 *q;
    const __nv_bfloat16 *bounds;
    const float *k_scale;      // E4M3 or null (its sign turns a key's bounds round)
    float2 *scores;            // [num_tokens][Hkv][score_stride]: score, sum of its terms' magnitudes
    int32_t score_stride;
    int32_t num_q_heads, num_kv_heads, group;
    int32_t num_selected, keep_first, keep_last;
    int32_t *selected;
};

// What the paged calls need of the context's workspace: two partial tiles per CTA (decode) or pair of CTAs
// (chunks) of the attention grid, or a score per (sequence, kv head, block) of max_batch single-token rows.
constexpr int64_t paged_partial_rows(int num_sms, bool chunk) {
    return chunk ? (int64_t)2 * (num_sms / 2) * kChunkRows : (int64_t)2 * kDecodeCtasPerSm * num_sms * kDecodeRows;
}
constexpr int64_t paged_partial_bytes(int num_sms) {
    return paged_partial_rows(num_sms, true) * (kHeadDim * 4 + 8);
}
static_assert(kChunkRows >= 2 * kDecodeCtasPerSm * kDecodeRows, "the chunk kernel's partials are the larger");
constexpr int64_t paged_rank_bytes(int64_t max_batch, int64_t num_kv_heads, int64_t max_context) {
    return max_batch * num_kv_heads * ((max_context >> kMinPageShift) + 1) * 8;
}

// Launch as a programmatic dependent of the previous kernel in the stream (each of these kernels waits for it
// before its first access to global memory), in clusters of `cluster` CTAs.
template <class... P, class... A>
cudaError_t launch_overlapping(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t s,
                               const A &...args) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim = {(unsigned)cluster, 1, 1};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_paged_append(const PagedAppendArgs &a, cudaStream_t s);
// kmap / vmap: 5-D views of the pages with boxes of min(page, stage) rows (paged_map_rows).
cudaError_t launch_paged_decode(const CUtensorMap *kmap, const CUtensorMap *vmap, const PagedAttnArgs &a, int num_sms,
                                cudaStream_t s);
// qmap: 4-D view {64 dims, heads, rows, 64-dim groups} of q_rot in boxes of group x 128 / group rows; kmap / vmap:
// boxes of chunk_k_rows / chunk_v_rows slots (paged_api.cpp).
cudaError_t launch_paged_chunk(const CUtensorMap *qmap, const CUtensorMap *kmap, const CUtensorMap *vmap,
                               const PagedAttnArgs &a, cudaStream_t s);
cudaError_t launch_paged_select(const PagedSelectArgs &a, int max_blocks, int num_sms, cudaStream_t s);

}  // namespace hd
