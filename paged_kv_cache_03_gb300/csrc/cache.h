// cache.h -- declarations shared by the translation units of the cache
// operators: 4-bit pages (append, read-back, attention), key weights and
// eviction.  Not part of the public ABI.
#pragma once
#include "internal.h"

namespace pa {

// Host-side check of the shape fields (PA_OK, PA_ERR_INVALID_ARG or
// PA_ERR_UNSUPPORTED).
pa_status check_shape(const pa_shape* s);

// A 4-bit row: 64 bytes of e2m1 codes and 8 e4m3 scales.
constexpr int kQ4CodeBytes = kHeadDim / 2;
constexpr int kQ4Groups = kHeadDim / 16;

pa_status q4_append_launch(const pa_shape& sh, const void* k_new, const void* v_new,
                           const pa_q4_pool& pool, const int32_t* bt, const int32_t* ctx,
                           uint32_t* flag, cudaStream_t stream);

// Dense rows [B, H_kv, n, D] (sh.dtype) of positions first + i, first = 0 or,
// with tail, context_lens[b] - n; outside [0, context_lens[b]) zeros, or with
// fill = 0 whatever was there.  id (or null) receives 0 .. B - 1, the block
// table under which the dense rows are a pool of B pages of n slots, and
// id + nid the lengths, 0 for one outside [0, capacity].
pa_status q4_gather_launch(const pa_shape& sh, const pa_q4_pool& pool, const int32_t* bt,
                           const int32_t* ctx, int n, int tail, int fill, int32_t* id, int nid,
                           void* k_dense, void* v_dense, uint32_t* flag, cudaStream_t stream);

// One attention call over 4-bit pages, or over bf16 pages with key weights.
struct WalkCall {
    pa_shape sh;
    const void* q;
    const void *kc, *vc;            // codes, or bf16 rows
    const void *ks, *vs;            // scales (4-bit pages), else null
    const int32_t* bt;
    const int32_t* ctx;
    float scale;
    int causal;
    void* out;
    const float* w_in;              // accumulated weights, or null (zeros)
    float* w_out;                   // or null: no weights
    long long w_S;
    void* ws;
    size_t ws_bytes;
    cudaStream_t stream;
    DeviceInfo dev;
};
// Enough for this shape and any with at most its B, L and max_pages_per_seq.
size_t walk_workspace_bytes(const pa_shape& sh, bool q4, bool weights, int sm_count);
pa_status walk_launch(const WalkCall& c);

// bf16 queries with many rows per kv head over 4-bit pages, on tcgen05 tiles
// (tiles.cu); lse: [B, H_q, L], or null.
bool tiles_supported(const pa_shape& sh, int sm_count);
size_t tiles_workspace_bytes(const pa_shape& sh, int sm_count);
size_t tiles_workspace_most(const pa_shape& sh, int sm_count);  // ... of any smaller call
pa_status tiles_launch(const WalkCall& c, float* lse);

// Eviction from the buffers K and V (rows of sh.dtype) or, where buf[2] is not
// null, K codes, V codes, K scales, V scales.
struct EvictCall {
    pa_shape sh;
    void* buf[4];
    const int32_t* bt;
    const int32_t* ctx;
    const float* w;
    long long w_S;
    int keep, recent;
    const int32_t* dst_bt;
    int dst_max_pages;
    int32_t* ctx_out;
    float* w_out;
    long long w_out_S;
    int32_t* kept;
    uint32_t* flag;
    cudaStream_t stream;
    DeviceInfo dev;
};
pa_status evict_launch(const EvictCall& c);

// Launches `kernel`, whose start may overlap the end of the kernel before it.
template <class... P, class... A>
inline bool launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

}  // namespace pa
