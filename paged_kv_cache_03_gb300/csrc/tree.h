// tree.h -- declarations shared by the translation units of draft trees
// (visibility, attention, compaction) and page sharing.  Not part of the public ABI.
#pragma once
#include "cache.h"

namespace pa {

constexpr int kTreeMax = 1024;  // drafted slots of a sequence at most
// Workspace: the CTAs-done counter of pa_resize_pages (zero between calls, among the other
// schedules' counters in the first 256 bytes).
constexpr size_t kPagesCounterOffset = 224;

inline int tree_words(int L) { return (L + 31) / 32; }

// One attention call of drafted trees over bf16 or fp32 pages (kc, vc) or, where ks is
// not null, 4-bit pages (codes kc, vc, scales ks, vs).
struct TreeCall {
    pa_shape sh;
    const void* q;
    const void *kc, *vc, *ks, *vs;
    const int32_t* bt;
    const int32_t* ctx;
    const uint32_t* mask;  // [B, L, words]
    float scale;
    void* out;
    void* ws;
    size_t ws_bytes;
    cudaStream_t stream;
    DeviceInfo dev;
};
bool tree_supported(const pa_shape& sh);
size_t tree_workspace_bytes(int sm_count);
pa_status tree_launch(const TreeCall& c);

pa_status tree_mask_launch(int B, int L, const int32_t* parents, uint32_t* mask, int32_t* depths, uint32_t* flag,
                           cudaStream_t stream);

// Row buffers of a pool: K and V rows of sh.dtype or, where buf[2] is not null, K codes,
// V codes, K scales, V scales.
struct PoolBufs {
    void* buf[4];
};

struct CompactCall {
    pa_shape sh;
    PoolBufs pool;
    const int32_t* bt;
    const int32_t* ctx;
    const int32_t* path;  // [B, path_n]
    int path_n;
    const int32_t* path_lens;
    int32_t* ctx_out;
    uint32_t* flag;
    cudaStream_t stream;
};
pa_status compact_launch(const CompactCall& c);

pa_status fork_launch(const pa_shape& sh, int32_t* bt, int32_t* ctx, int32_t* refs, const int32_t* sources,
                      const int32_t* targets, const int32_t* lens, int n, uint32_t* flag, cudaStream_t stream);
size_t pages_workspace_bytes(const pa_shape& sh);
pa_status resize_launch(const pa_shape& sh, int32_t* bt, int32_t* ctx, int32_t* refs, const int32_t* new_lens,
                        int32_t* copies, void* ws, int sm_count, cudaStream_t stream);
pa_status copy_pages_launch(const pa_shape& sh, const PoolBufs& pool, const int32_t* copies, int n, uint32_t* flag,
                            cudaStream_t stream);

}  // namespace pa
