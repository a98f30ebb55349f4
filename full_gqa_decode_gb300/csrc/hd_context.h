// The context behind hd_ctx and the host helpers that the API files share.
// Not part of the C ABI.
#pragma once

#include <cudaTypedefs.h>

#include <cstdint>
#include <mutex>
#include <vector>

#include "hd_internal.h"

namespace hd {

struct MapCacheEntry {
    const void *k = nullptr, *v = nullptr;
    int64_t seq_stride = 0;
    int32_t capacity = 0, batch = 0;
    CUtensorMap kmap, vmap;     // boxes of one stage's keys
    bool wide_valid = false;    // kmapw / vmapw encoded for this cache
    CUtensorMap kmapw, vmapw;   // boxes of kWideBoxRows keys (64-key bf16 stages)
};

struct DeviceTable {
    float2 *data = nullptr;  // [max_context + 1][rotary_dim / 2]
    int32_t rotary_dim = 0;
};

// Launches the fused layer kernel (see attn_decode.cu) for one layer call.
struct LayerCall {
    int layer, batch;
    const int32_t *context;
    int max_keys;           // bound on the cached keys any sequence scores (split plan)
    int key_set, new_kind, commit;
    const void *q_bf16;     // rotate q in the kernel, or
    const float *q_rot;     // take it rotated
    const void *new_k, *new_v;
    hd_kv_cache cache;
    const float *sink;
    const float *gate;
    void *out;
    float *lse;
    bool pdl;               // previous grid in the stream is this step's previous layer kernel
    bool early = false;     // pdl: the layer may read and stream before that grid completes
    bool one_chunk = false; // step grids: the layer needs a single chunk per sequence
    int tokens = 1, token0 = 0, total_tokens = 1;   // multi-token decode: this pass's tokens
};

}  // namespace hd

struct hd_ctx {
    hd_config cfg;
    std::vector<int32_t> layer_types;
    int device = 0;
    int num_sms = 0;
    int group = 1;
    int sliding_layout = HD_LAYOUT_RING;
    hd::DeviceTable table_sliding, table_full;
    float *part_o = nullptr;
    float2 *part_ml = nullptr;
    int64_t part_slots = 0;              // single-layer calls: capacity in (sequence, chunk) pairs
    int64_t part_rows = 0;               // capacity in partial rows ([256] floats + (m, l) each)
    // Paged calls take part_o as bytes: partial rows and (m, l) of cut items, or scores of blocks.
    uint8_t *paged_ws() const { return reinterpret_cast<uint8_t *>(part_o); }
    int64_t paged_ws_bytes() const { return part_rows * hd::kHeadDim * (int64_t)sizeof(float); }
    uint8_t *stage_k = nullptr;          // [num_layers][max_batch][Hkv][D] entries of the cache type
    uint8_t *stage_v = nullptr;
    int kv_type = hd::KV_BF16;
    int32_t *counters = nullptr;         // [num_layers][max_batch][Hkv] chunk tickets, zero between calls
    int32_t *err = nullptr;
    int32_t *paged_tickets = nullptr;    // [kPagedTickets], zero between calls
    int consumer = hd::CONSUMER_MMA;
    int cluster_max = 0;                 // largest cluster the single-layer kernel runs with (0: none)
    bool cluster_combine = true;         // single-layer calls: small grids merge chunks in a cluster
    int32_t drop_stage = -1;             // test hook, see hybrid_decode_inject_lost_copy
    bool layer_overlap = true;           // decode_step: layers start before the previous one finishes
    bool fuse_step = true;               // decode_step: one grid for all layers (step tables)
    hd::StepTable step_table;                // parameters of the step grid being launched
    std::vector<hd::LayerCall> step_calls;   // the layer calls of the step being launched
    std::vector<int> step_order;         // their order in the step grids
    // Last independence check of decode_step's layers (host memcmp of the array).
    std::vector<hd_layer_io> indep_layers;
    int32_t indep_batch = -1, indep_tokens = -1;
    bool indep_ok = false;
    int64_t launches = 0;
    std::vector<hd::MapCacheEntry> maps;     // one per layer
    int32_t profile_mask = 0;           // bit (1 << layer type): bracket that type's launches
    bool profile_seen[2] = {false, false};  // FIRST_ONLY: a layer of that type was bracketed in this step
    std::vector<cudaEvent_t> ev_begin, ev_end;  // [3][kProfileEvents]: per layer type, then step grids
    size_t ev_used[3] = {0, 0, 0};
};

namespace hd {

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }


// The context's workspace and tensor maps live on the device it was created on.
inline hd_status check_device(const hd_ctx *ctx) {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && dev == ctx->device ? HD_OK : HD_ERR_STATE;
}

inline hd_status cuda_status(cudaError_t e) { return e == cudaSuccess ? HD_OK : HD_ERR_CUDA; }

}  // namespace hd
