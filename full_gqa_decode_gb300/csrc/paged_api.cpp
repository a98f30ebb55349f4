// Host side of the paged-cache entry points of include/hybrid_decode.h:
// argument checks, tensor maps and launches.
#include "paged.h"

#include <algorithm>
#include <climits>
#include <cmath>

#include "hd_context.h"

using namespace hd;

namespace {

constexpr float kLog2e = 1.4426950408889634f;

bool page_shift_of(int page_size, int *shift) {
    for (int s = kMinPageShift; s <= kMaxPageShift; ++s)
        if (page_size == 1 << s) {
            *shift = s;
            return true;
        }
    return false;
}

// Checks shared by all paged calls; fills the sequences' kernel arguments.
hd_status check_paged(const hd_ctx *ctx, int layer, const hd_paged_batch *b, const hd_paged_cache *c, PagedSeqs *s) {
    if (!ctx || layer < 0 || layer >= ctx->cfg.num_layers) return HD_ERR_INVALID_ARG;
    const hd_status st = hd_validate_paged(&ctx->cfg, b, c);
    if (st != HD_OK) return st;
    int shift = 0;
    page_shift_of(c->page_size, &shift);
    *s = PagedSeqs{};
    s->table = b->block_table;
    s->table_stride = b->table_stride;
    s->context = b->context;
    s->offsets = b->token_offsets;
    s->batch = b->batch;
    s->num_tokens = b->num_tokens;
    s->max_tokens = b->max_tokens;
    s->max_blocks = b->max_blocks;
    s->max_context = b->max_context ? b->max_context : ctx->cfg.max_context;   // seq_span looks at context + tokens too
    s->max_position = ctx->cfg.max_context;
    s->page_shift = shift;
    s->num_pages = c->num_pages;
    s->err = ctx->err;
    return check_device(ctx);
}

// 5-D view {128 bytes of dims, slots, 128-byte column groups, kv heads, pages} of a pool's k or v, read in
// boxes of `rows` slots x `groups` column groups, which land as column groups of `rows` swizzled 128-byte rows.
// Page number num_pages lies outside: a copy of it fills zeros.
bool encode_pages(CUtensorMap *map, const void *base, const hd_paged_cache &c, int num_kv_heads, int kv_type, int rows,
                  int groups) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t es = (cuuint64_t)kv_elem_bytes(kv_type);
    const cuuint64_t cols = (cuuint64_t)kv_box_cols(kv_type), all = (cuuint64_t)kv_boxes_per_row(kv_type);
    const cuuint64_t dims[5] = {cols, (cuuint64_t)c.page_size, all, (cuuint64_t)num_kv_heads, (cuuint64_t)c.num_pages};
    const cuuint64_t strides[4] = {kHeadDim * es, 128, (cuuint64_t)c.page_size * kHeadDim * es,
                                   (cuuint64_t)c.page_stride * es};
    const cuuint32_t box[5] = {(cuuint32_t)cols, (cuuint32_t)rows, (cuuint32_t)groups, 1, 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return fn(map, kv_type == KV_FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
              const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 4-D view {64 dims, query heads, rows, 64-dim groups} of the rotated queries in boxes of one kv head's heads x as
// many tokens as make 128 rows; rows behind the last fill zeros.
bool encode_queries(CUtensorMap *map, const void *q, int num_q_heads, int num_tokens, int group) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {64, (cuuint64_t)num_q_heads, (cuuint64_t)num_tokens, kHeadDim / 64};
    const cuuint64_t strides[3] = {kHeadDim * 2, (cuuint64_t)num_q_heads * kHeadDim * 2, 128};
    const cuuint32_t box[4] = {64, (cuuint32_t)group, (cuuint32_t)(kChunkRows / 2 / group), kHeadDim / 64};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(q), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether the decode kernel serves a call with more rows per kv head than its tiles hold sooner than the chunk kernel: it reads
// a sequence's keys once per eight rows, the chunk kernel once per 256 rows, but with a longer start and drain.  Estimates in
// microseconds, fitted to calls of 1 to 256 sequences with 12 to 160 rows each behind 0 to 30000 keys; they pick the slower
// kernel by more than 8 % in 3 of 140, given exact bounds (a max_context of 0 is taken for the whole capacity).  Measured
// decode and chunk: 2 to 7 tokens of 16 sequences in 512-key windows 15.7 and 24.4 us; 16 tokens of one sequence at 8000 27.8
// and 42.4; 7 tokens of 16 sequences at 8000 158 and 74; 3 tokens of 64 at 8000 over E4M3 pages 170 and 342.
constexpr int kDecodeRowsMost = 160;
bool decode_is_sooner(const hd_ctx *ctx, const PagedSeqs &s, int window) {
    const int64_t rows = (int64_t)s.max_tokens * ctx->group;
    if (rows <= kDecodeRows || rows > kDecodeRowsMost) return rows <= kDecodeRows;
    int64_t keys = std::min({(int64_t)s.max_context + s.max_tokens, (int64_t)s.max_position + 1,
                             (int64_t)s.max_blocks << s.page_shift});
    if (window) keys = std::min(keys, (int64_t)window - 1 + s.max_tokens);
    // Tiles of the call in each kernel: by the longest sequence, or by all its rows.
    const auto items = [&](int64_t tile) {
        const int64_t all = (int64_t)s.num_tokens * ctx->group / tile + s.batch;
        return (double)std::min(s.batch * ((rows + tile - 1) / tile), all) * ctx->cfg.num_kv_heads;
    };
    const bool fp8 = ctx->kv_type == KV_FP8;
    const double units = keys / 128.0, few = items(kDecodeRows), wide = items(kChunkRows), pairs = ctx->num_sms / 2;
    const double decode = 10.0 + few * ((fp8 ? 0.0098 : 0.018) * units + 0.01);
    const double pieces = std::min(pairs / wide, units / 4);   // of an item, which are merged
    return decode < (fp8 ? 28.0 : 20.0) + (fp8 ? 0.039 : 0.0263) * wide * (units + 2) + 0.6 * pieces;
}

hd_status attend(hd_ctx *ctx, int layer, const PagedSeqs &seqs, const void *q_rot, const hd_paged_cache &c,
                 const int32_t *selected, int num_selected, const hd_scoring *rule, const float *sink, const float *gate,
                 void *out, float *lse, void *stream) {
    if (seqs.num_tokens == 0) return HD_OK;   // no rows: their tensors may be null
    if (!q_rot || !aligned16(q_rot) || !out || !aligned16(out) || !lse) return HD_ERR_INVALID_ARG;
    PagedAttnArgs a{};
    a.seqs = seqs;
    a.q = static_cast<const __nv_bfloat16 *>(q_rot);
    a.selected = selected;
    a.num_selected = num_selected;
    a.k_codes = static_cast<const uint8_t *>(c.k);
    a.v_codes = static_cast<const uint8_t *>(c.v);
    a.page_stride = c.page_stride;
    a.k_scale = c.k_scale;
    a.v_scale = c.v_scale;
    a.sink = sink;
    a.gate = gate;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.tickets = ctx->paged_tickets;
    a.num_q_heads = ctx->cfg.num_q_heads;
    a.num_kv_heads = ctx->cfg.num_kv_heads;
    a.group = ctx->group;
    while (1 << a.group_shift < a.group) ++a.group_shift;
    a.window = ctx->layer_types[layer] == HD_SLIDING ? ctx->cfg.sliding_window : 0;
    a.kv_type = ctx->kv_type;
    a.drop_stage = ctx->drop_stage;
    if (rule) {
        a.scored = 1;
        a.qscale = (rule->scale != 0.f ? rule->scale : 1.f / 16.f) * kLog2e;
        if (rule->softcap != 0.f) {
            a.cap = rule->softcap * kLog2e;
            a.two_over_cap = 2.f / rule->softcap;
        }
        a.slopes = rule->slopes;
        a.first = rule->first;
        a.last = rule->last;
    }
    // More than eight rows per kv head in some sequence: the tensor-memory kernel, which also serves the call's
    // single tokens (with a rule, unless the decode kernel is sooner); lists of selected blocks are the decode kernel's (each token and kv head has its own keys).
    const bool few = rule ? decode_is_sooner(ctx, seqs, a.window) : (int64_t)seqs.max_tokens * ctx->group <= kDecodeRows;
    const bool chunk = !selected && !few;
    const int64_t rows = paged_partial_rows(ctx->num_sms, chunk);
    a.part_o = reinterpret_cast<float *>(ctx->paged_ws());
    a.part_ml = reinterpret_cast<float2 *>(ctx->paged_ws() + rows * kHeadDim * 4);
    const int Hkv = ctx->cfg.num_kv_heads, all = kv_boxes_per_row(ctx->kv_type), ps = c.page_size;
    const bool fp8 = ctx->kv_type == KV_FP8;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CUtensorMap km{}, vm{}, qm{};
    hd_status st;
    if (chunk) {
        const int krows = std::min(ps, kChunkKeys / 2), vrows = std::min(ps, kChunkKeys);
        const int kgroups = krows == kChunkKeys / 2 ? all : 1;
        if ((!fp8 && (!encode_pages(&km, c.k, c, Hkv, ctx->kv_type, krows, kgroups) ||
                      !encode_pages(&vm, c.v, c, Hkv, ctx->kv_type, vrows, all / 2))) ||
            !encode_queries(&qm, q_rot, ctx->cfg.num_q_heads, seqs.num_tokens, ctx->group))
            return HD_ERR_CUDA;
        st = cuda_status(launch_paged_chunk(&qm, &km, &vm, a, s));
    } else {
        const int box = std::min(ps, kv_stage_keys(ctx->kv_type));
        if (!encode_pages(&km, c.k, c, Hkv, ctx->kv_type, box, all) ||
            !encode_pages(&vm, c.v, c, Hkv, ctx->kv_type, box, all))
            return HD_ERR_CUDA;
        st = cuda_status(launch_paged_decode(&km, &vm, a, ctx->num_sms, s));
    }
    if (st == HD_OK) ++ctx->launches;
    return st;
}

// Checks of an append's tensors; fills everything of its kernel arguments but the angles.
hd_status check_append(const hd_ctx *ctx, int layer, const hd_paged_batch *batch, const void *q, int64_t q_stride, const void *k,
                       int64_t k_stride, const void *v, int64_t v_stride, void *q_rot, const hd_paged_cache *cache,
                       PagedAppendArgs *out) {
    PagedAppendArgs &a = *out;
    const hd_status st = check_paged(ctx, layer, batch, cache, &a.seqs);
    if (st != HD_OK || batch->num_tokens == 0) return st;
    const int64_t Hq = ctx->cfg.num_q_heads, Hkv = ctx->cfg.num_kv_heads;
    if (!k || !v || !aligned16(k) || !aligned16(v) || (q == nullptr) != (q_rot == nullptr) || !aligned16(q) ||
        !aligned16(q_rot))
        return HD_ERR_INVALID_ARG;
    if (k_stride % 8 || v_stride % 8 || k_stride < Hkv * kHeadDim || v_stride < Hkv * kHeadDim ||
        (q && (q_stride % 8 || q_stride < Hq * kHeadDim)))
        return HD_ERR_INVALID_ARG;
    // q_rot in place of q, row by row, or apart from it: elsewhere its rows would lie over rows not yet rotated.
    const auto *src = static_cast<const uint8_t *>(q), *dst = static_cast<const uint8_t *>(q_rot);
    const int64_t row = Hq * kHeadDim * 2, rows = batch->num_tokens;
    if (q && src < dst + rows * row && dst < src + (rows - 1) * q_stride * 2 + row &&
        !(src == dst && (rows == 1 || q_stride == Hq * kHeadDim)))
        return HD_ERR_INVALID_ARG;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.v = static_cast<const __nv_bfloat16 *>(v);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_rot = static_cast<__nv_bfloat16 *>(q_rot);
    a.cache_k = cache->k;
    a.cache_v = cache->v;
    a.page_stride = cache->page_stride;
    a.k_scale = cache->k_scale;
    a.v_scale = cache->v_scale;
    a.bounds = static_cast<__nv_bfloat16 *>(cache->bounds);
    a.num_q_heads = (int32_t)Hq;
    a.num_kv_heads = (int32_t)Hkv;
    a.kv_type = ctx->kv_type;
    return HD_OK;
}

}  // namespace

extern "C" {

hd_status hd_validate_paged(const hd_config *cfg, const hd_paged_batch *b, const hd_paged_cache *c) {
    hd_status st = hd_validate_config(cfg);
    if (st != HD_OK) return st;
    if (!b || !c || !b->block_table || !b->context) return HD_ERR_INVALID_ARG;
    if (b->batch <= 0 || b->num_tokens < 0 || b->max_tokens <= 0 || b->max_context < 0 || b->max_blocks <= 0 ||
        b->table_stride < b->max_blocks)
        return HD_ERR_INVALID_ARG;
    if (!b->token_offsets && (b->num_tokens != b->batch || b->max_tokens != 1)) return HD_ERR_INVALID_ARG;
    int shift = 0;
    if (!page_shift_of(c->page_size, &shift)) return HD_ERR_UNSUPPORTED;
    const int es = kv_elem_bytes(cfg->kv_dtype == HD_KV_FP8_E4M3 ? KV_FP8 : KV_BF16);
    const int64_t page = (int64_t)cfg->num_kv_heads * c->page_size * kHeadDim;
    if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v) || !aligned16(c->bounds)) return HD_ERR_INVALID_ARG;
    if (c->num_pages <= 0 || c->num_pages == INT_MAX || c->page_stride < page || (c->page_stride * es) % 16 != 0)
        return HD_ERR_INVALID_ARG;
    const bool fp8 = cfg->kv_dtype == HD_KV_FP8_E4M3;
    if (fp8 != (c->k_scale != nullptr) || fp8 != (c->v_scale != nullptr)) return HD_ERR_INVALID_ARG;
    if (b->batch > cfg->max_batch || b->max_context > cfg->max_context) return HD_ERR_CAPACITY;
    return HD_OK;
}

hd_status rope_append_paged(hd_ctx *ctx, int32_t layer, const hd_paged_batch *batch, const void *q, int64_t q_stride,
                            const void *k, int64_t k_stride, const void *v, int64_t v_stride, void *q_rot,
                            const hd_paged_cache *cache, void *stream) {
    PagedAppendArgs a{};
    hd_status st = check_append(ctx, layer, batch, q, q_stride, k, k_stride, v, v_stride, q_rot, cache, &a);
    if (st != HD_OK || batch->num_tokens == 0) return st;
    const DeviceTable &tab = ctx->layer_types[layer] == HD_SLIDING ? ctx->table_sliding : ctx->table_full;
    if (tab.rotary_dim % 8) return HD_ERR_UNSUPPORTED;
    a.rope = tab.data;
    a.rotary_dim = tab.rotary_dim;
    st = cuda_status(launch_paged_append(a, static_cast<cudaStream_t>(stream)));
    if (st == HD_OK) ++ctx->launches;
    return st;
}

hd_status norm_rope_append_paged(hd_ctx *ctx, int32_t layer, const hd_paged_batch *batch, const hd_head_norm *norm,
                                 const hd_rope_table *rope, const int32_t *positions, const void *q, int64_t q_stride,
                                 const void *k, int64_t k_stride, const void *v, int64_t v_stride, void *q_rot,
                                 const hd_paged_cache *cache, void *stream) {
    PagedNormArgs a{};
    hd_status st = check_append(ctx, layer, batch, q, q_stride, k, k_stride, v, v_stride, q_rot, cache, &a.entry);
    if (st != HD_OK) return st;
    if (norm && (!aligned16(norm->q_weight) || !aligned16(norm->k_weight) || !std::isfinite(norm->offset) || !(norm->eps > 0.f) ||
                 !std::isfinite(norm->eps)))
        return HD_ERR_INVALID_ARG;
    if (rope && (!rope->table || !aligned16(rope->table) || rope->positions < 1 || rope->rotary_dim < 8 ||
                 rope->rotary_dim > kHeadDim || rope->rotary_dim % 8 || rope->layout < HD_ROPE_HALVES ||
                 rope->layout > HD_ROPE_NEIGHBOURS))
        return HD_ERR_INVALID_ARG;
    if (batch->num_tokens == 0) return HD_OK;
    if (rope) {
        a.entry.rope = reinterpret_cast<const float2 *>(rope->table);
        a.entry.rotary_dim = rope->rotary_dim;
        a.table_rows = rope->positions;
        a.neighbours = rope->layout == HD_ROPE_NEIGHBOURS;
    } else {
        const DeviceTable &tab = ctx->layer_types[layer] == HD_SLIDING ? ctx->table_sliding : ctx->table_full;
        if (tab.rotary_dim % 8) return HD_ERR_UNSUPPORTED;
        a.entry.rope = tab.data;
        a.entry.rotary_dim = tab.rotary_dim;
        a.table_rows = ctx->cfg.max_context + 1;
    }
    a.positions = positions;
    if (!positions) a.entry.seqs.max_position = std::min(a.entry.seqs.max_position, a.table_rows - 1);
    if (norm) {
        a.norm = 1;
        a.q_weight = norm->q_weight;
        a.k_weight = norm->k_weight;
        a.f32_weights = norm->f32_weights != 0;
        a.per_head = norm->per_head != 0;
        a.offset = norm->offset;
        a.eps = norm->eps;
    }
    st = cuda_status(launch_paged_norm_append(a, static_cast<cudaStream_t>(stream)));
    if (st == HD_OK) ++ctx->launches;
    return st;
}

hd_status read_paged(hd_ctx *ctx, const hd_paged_batch *batch, const hd_paged_cache *cache, void *k, int64_t k_stride, void *v,
                     int64_t v_stride, void *stream) {
    PagedReadArgs a{};
    hd_status st = check_paged(ctx, 0, batch, cache, &a.seqs);
    if (st != HD_OK || batch->num_tokens == 0 || (!k && !v)) return st;
    const int64_t row = (int64_t)ctx->cfg.num_kv_heads * kHeadDim;
    if (!aligned16(k) || !aligned16(v) || (k && (k_stride % 8 || k_stride < row)) || (v && (v_stride % 8 || v_stride < row)))
        return HD_ERR_INVALID_ARG;
    a.cache_k = cache->k;
    a.cache_v = cache->v;
    a.page_stride = cache->page_stride;
    a.k_scale = cache->k_scale;
    a.v_scale = cache->v_scale;
    a.k = static_cast<__nv_bfloat16 *>(k);
    a.v = static_cast<__nv_bfloat16 *>(v);
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.num_kv_heads = ctx->cfg.num_kv_heads;
    a.kv_type = ctx->kv_type;
    st = cuda_status(launch_paged_read(a, static_cast<cudaStream_t>(stream)));
    if (st == HD_OK) ++ctx->launches;
    return st;
}

hd_status attn_paged_scored(hd_ctx *ctx, int32_t layer, const hd_paged_batch *batch, const hd_scoring *scoring,
                            const void *q_rot, const hd_paged_cache *cache, const float *sink, const float *gate, void *out,
                            float *lse, void *stream) {
    PagedSeqs s;
    const hd_status st = check_paged(ctx, layer, batch, cache, &s);
    if (st != HD_OK) return st;
    if (scoring) {
        const float scale = scoring->scale, cap = scoring->softcap;
        if (!std::isfinite(scale) || scale < 0.f || !std::isfinite(cap) || cap < 0.f) return HD_ERR_INVALID_ARG;
        if ((cap != 0.f && (cap < 1.f / 1024.f || cap > 1024.f)) || (scale != 0.f && (scale < 0x1p-32f || scale > 0x1p32f)))
            return HD_ERR_UNSUPPORTED;
    }
    return attend(ctx, layer, s, q_rot, *cache, nullptr, 0, scoring, sink, gate, out, lse, stream);
}

hd_status attn_paged(hd_ctx *ctx, int32_t layer, const hd_paged_batch *batch, const void *q_rot,
                     const hd_paged_cache *cache, const float *sink, const float *gate, void *out, float *lse,
                     void *stream) {
    PagedSeqs s;
    const hd_status st = check_paged(ctx, layer, batch, cache, &s);
    if (st != HD_OK) return st;
    return attend(ctx, layer, s, q_rot, *cache, nullptr, 0, nullptr, sink, gate, out, lse, stream);
}

hd_status select_pages(hd_ctx *ctx, int32_t layer, const hd_paged_batch *batch, const void *q_rot,
                       const hd_paged_cache *cache, int32_t num_selected, int32_t keep_first, int32_t keep_last,
                       int32_t *selected, void *stream) {
    PagedSelectArgs a{};
    hd_status st = check_paged(ctx, layer, batch, cache, &a.seqs);
    if (st != HD_OK) return st;
    if (ctx->layer_types[layer] != HD_FULL) return HD_ERR_STATE;
    if (!cache->bounds || num_selected < 1 || keep_first < 0 || keep_last < 0 ||
        (int64_t)keep_first + keep_last > num_selected)
        return HD_ERR_INVALID_ARG;
    if (batch->num_tokens == 0) return HD_OK;
    if (!q_rot || !aligned16(q_rot) || !selected) return HD_ERR_INVALID_ARG;
    const int64_t last = std::min<int64_t>((int64_t)a.seqs.max_context + batch->max_tokens - 1, ctx->cfg.max_context);
    const int64_t blocks = std::min<int64_t>((last >> a.seqs.page_shift) + 1, batch->max_blocks);
    if (blocks > kMaxSelectBlocks ||
        (int64_t)batch->num_tokens * ctx->cfg.num_kv_heads * blocks * 8 > ctx->paged_ws_bytes())
        return HD_ERR_CAPACITY;
    a.q = static_cast<const __nv_bfloat16 *>(q_rot);
    a.bounds = static_cast<const __nv_bfloat16 *>(cache->bounds);
    a.k_scale = cache->k_scale;
    a.scores = reinterpret_cast<float2 *>(ctx->paged_ws());
    a.score_stride = (int32_t)blocks;
    a.num_q_heads = ctx->cfg.num_q_heads;
    a.num_kv_heads = ctx->cfg.num_kv_heads;
    a.group = ctx->group;
    a.num_selected = num_selected;
    a.keep_first = keep_first;
    a.keep_last = keep_last;
    a.selected = selected;
    st = cuda_status(launch_paged_select(a, (int)blocks, ctx->num_sms, static_cast<cudaStream_t>(stream)));
    if (st == HD_OK) ctx->launches += 2;
    return st;
}

hd_status attn_selected_pages(hd_ctx *ctx, int32_t layer, const hd_paged_batch *batch, const void *q_rot,
                              const hd_paged_cache *cache, const int32_t *selected, int32_t num_selected,
                              const float *sink, const float *gate, void *out, float *lse, void *stream) {
    PagedSeqs s;
    const hd_status st = check_paged(ctx, layer, batch, cache, &s);
    if (st != HD_OK) return st;
    if (ctx->layer_types[layer] != HD_FULL) return HD_ERR_STATE;
    if ((!selected && batch->num_tokens) || num_selected < 1) return HD_ERR_INVALID_ARG;
    return attend(ctx, layer, s, q_rot, *cache, selected, num_selected, nullptr, sink, gate, out, lse, stream);
}

}  // extern "C"
