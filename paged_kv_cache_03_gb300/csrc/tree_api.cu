// tree_api.cu -- the extern "C" entry points of draft trees and page sharing.
// Argument checks on the host, then the launches.
#include <climits>

#include "tree.h"

namespace pa {
namespace {

bool on(const void* p, uintptr_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }

bool pool_ok(const pa_q4_pool* p) {
    return p && on(p->key_codes, 16) && on(p->value_codes, 16) && on(p->key_scales, 16) && on(p->value_scales, 16);
}

pa_status device_ok(DeviceInfo* dev) {
    const pa_status st = current_device_info(dev);
    if (st != PA_OK) return st;
    return dev->cc_major == 10 && dev->cc_minor == 3 ? PA_OK : PA_ERR_UNSUPPORTED;
}

PoolBufs bufs(const pa_q4_pool& p) { return {{p.key_codes, p.value_codes, p.key_scales, p.value_scales}}; }

pa_status attend(const pa_shape* shape, const void* query, const void* kc, const void* vc, const void* ks,
                 const void* vs, const int32_t* bt, const int32_t* ctx, const uint32_t* mask, float scale, void* out,
                 void* ws, size_t ws_bytes, void* stream) {
    pa_status st = check_call_args(shape, query, kc, vc, bt, ctx, scale, out);
    if (st != PA_OK) return st;
    if (!on(mask, 4)) return PA_ERR_INVALID_ARG;
    if (!tree_supported(*shape)) return PA_ERR_UNSUPPORTED;
    if (!on(ws, 256)) return PA_ERR_WORKSPACE;
    TreeCall c;
    st = device_ok(&c.dev);
    if (st != PA_OK) return st;
    if (ws_bytes < tree_workspace_bytes(c.dev.sm_count)) return PA_ERR_WORKSPACE;
    c.sh = *shape;
    c.q = query;
    c.kc = kc;
    c.vc = vc;
    c.ks = ks;
    c.vs = vs;
    c.bt = bt;
    c.ctx = ctx;
    c.mask = mask;
    c.scale = scale;
    c.out = out;
    c.ws = ws;
    c.ws_bytes = ws_bytes;
    c.stream = static_cast<cudaStream_t>(stream);
    return tree_launch(c);
}

pa_status compact(const pa_shape* shape, const PoolBufs& pool, const int32_t* bt, const int32_t* ctx, const int32_t* path,
                  int path_n, const int32_t* path_lens, int32_t* ctx_out, void* ws, size_t ws_bytes, void* stream) {
    if (!on(bt, 4) || !on(ctx, 4) || !on(path, 4) || !on(path_lens, 4) || !on(ctx_out, 4) || path_n < 1 || ctx_out == ctx)
        return PA_ERR_INVALID_ARG;
    if (!on(ws, 4) || ws_bytes < kFlagBytes) return PA_ERR_WORKSPACE;
    DeviceInfo dev;
    const pa_status st = device_ok(&dev);
    if (st != PA_OK) return st;
    return compact_launch({*shape, pool, bt, ctx, path, path_n, path_lens, ctx_out, static_cast<uint32_t*>(ws),
                           static_cast<cudaStream_t>(stream)});
}

pa_status copy(const pa_shape* shape, const PoolBufs& pool, const int32_t* copies, int n, void* ws, size_t ws_bytes,
               void* stream) {
    if (n == 0) return PA_OK;  // (nothing of an empty list is read)
    if (!on(copies, 4) || n < 0) return PA_ERR_INVALID_ARG;
    if (!on(ws, 4) || ws_bytes < kFlagBytes) return PA_ERR_WORKSPACE;
    DeviceInfo dev;
    const pa_status st = device_ok(&dev);
    if (st != PA_OK) return st;
    return copy_pages_launch(*shape, pool, copies, n, static_cast<uint32_t*>(ws), static_cast<cudaStream_t>(stream));
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

pa_status pa_tree_mask(int B, int L, const int32_t* parents, uint32_t* mask, int32_t* depths, void* workspace,
                       size_t workspace_bytes, void* cuda_stream) {
    if (B < 1 || L < 1 || !on(parents, 4) || !on(mask, 4) || !on(depths, 4)) return PA_ERR_INVALID_ARG;
    if (L > kTreeMax) return PA_ERR_UNSUPPORTED;
    if (!on(workspace, 4) || workspace_bytes < kFlagBytes) return PA_ERR_WORKSPACE;
    DeviceInfo dev;
    const pa_status st = device_ok(&dev);
    if (st != PA_OK) return st;
    return tree_mask_launch(B, L, parents, mask, depths, static_cast<uint32_t*>(workspace),
                            static_cast<cudaStream_t>(cuda_stream));
}

size_t pa_tree_workspace_bytes(const pa_shape* shape) {
    DeviceInfo dev;
    if (check_shape(shape) != PA_OK || !tree_supported(*shape) || current_device_info(&dev) != PA_OK) return 0;
    return tree_workspace_bytes(dev.sm_count);
}

pa_status pa_paged_attention_tree(const pa_shape* shape, const void* query, const void* key_pages,
                                  const void* value_pages, const int32_t* block_table, const int32_t* context_lens,
                                  const uint32_t* tree_mask, float scale, void* out, void* workspace,
                                  size_t workspace_bytes, void* cuda_stream) {
    return attend(shape, query, key_pages, value_pages, nullptr, nullptr, block_table, context_lens, tree_mask, scale,
                  out, workspace, workspace_bytes, cuda_stream);
}

pa_status pa_paged_attention_tree_q4(const pa_shape* shape, const void* query, const pa_q4_pool* pool,
                                     const int32_t* block_table, const int32_t* context_lens, const uint32_t* tree_mask,
                                     float scale, void* out, void* workspace, size_t workspace_bytes, void* cuda_stream) {
    const pa_status st = check_shape(shape);
    if (st != PA_OK) return st;
    if (!pool_ok(pool)) return PA_ERR_INVALID_ARG;
    return attend(shape, query, pool->key_codes, pool->value_codes, pool->key_scales, pool->value_scales, block_table,
                  context_lens, tree_mask, scale, out, workspace, workspace_bytes, cuda_stream);
}

pa_status pa_compact_kv(const pa_shape* shape, void* key_pages, void* value_pages, const int32_t* block_table,
                        const int32_t* context_lens, const int32_t* path, int path_n, const int32_t* path_lens,
                        int32_t* context_lens_out, void* workspace, size_t workspace_bytes, void* cuda_stream) {
    const pa_status st = check_shape(shape);
    if (st != PA_OK) return st;
    if (!on(key_pages, 16) || !on(value_pages, 16)) return PA_ERR_INVALID_ARG;
    return compact(shape, {{key_pages, value_pages, nullptr, nullptr}}, block_table, context_lens, path, path_n, path_lens,
                   context_lens_out, workspace, workspace_bytes, cuda_stream);
}

pa_status pa_compact_kv_q4(const pa_shape* shape, const pa_q4_pool* pool, const int32_t* block_table,
                           const int32_t* context_lens, const int32_t* path, int path_n, const int32_t* path_lens,
                           int32_t* context_lens_out, void* workspace, size_t workspace_bytes, void* cuda_stream) {
    const pa_status st = check_shape(shape);
    if (st != PA_OK) return st;
    if (!pool_ok(pool)) return PA_ERR_INVALID_ARG;
    return compact(shape, bufs(*pool), block_table, context_lens, path, path_n, path_lens, context_lens_out, workspace,
                   workspace_bytes, cuda_stream);
}

size_t pa_pages_workspace_bytes(const pa_shape* shape) {
    return check_shape(shape) == PA_OK ? pages_workspace_bytes(*shape) : 0;
}

pa_status pa_fork_pages(const pa_shape* shape, int32_t* block_table, int32_t* context_lens, int32_t* page_refs,
                        const int32_t* sources, const int32_t* targets, const int32_t* lens, int n, void* workspace,
                        size_t workspace_bytes, void* cuda_stream) {
    pa_status st = check_shape(shape);
    if (st != PA_OK) return st;
    if (n == 0) return PA_OK;  // (nothing of an empty list is read)
    if (!on(block_table, 4) || !on(context_lens, 4) || !on(page_refs, 4) || !on(sources, 4) || !on(targets, 4) || n < 0 ||
        (lens && !on(lens, 4)))
        return PA_ERR_INVALID_ARG;
    if (!on(workspace, 4) || workspace_bytes < kFlagBytes) return PA_ERR_WORKSPACE;
    DeviceInfo dev;
    st = device_ok(&dev);
    if (st != PA_OK) return st;
    return fork_launch(*shape, block_table, context_lens, page_refs, sources, targets, lens, n,
                       static_cast<uint32_t*>(workspace), static_cast<cudaStream_t>(cuda_stream));
}

pa_status pa_resize_pages(const pa_shape* shape, int32_t* block_table, int32_t* context_lens, int32_t* page_refs,
                          const int32_t* new_lens, int32_t* copies, void* workspace, size_t workspace_bytes,
                          void* cuda_stream) {
    pa_status st = check_shape(shape);
    if (st != PA_OK) return st;
    if (!on(block_table, 4) || !on(context_lens, 4) || !on(page_refs, 4) || !on(new_lens, 4) || !on(copies, 4) ||
        new_lens == context_lens)
        return PA_ERR_INVALID_ARG;
    if (!on(workspace, 256) || workspace_bytes < pages_workspace_bytes(*shape)) return PA_ERR_WORKSPACE;
    DeviceInfo dev;
    st = device_ok(&dev);
    if (st != PA_OK) return st;
    return resize_launch(*shape, block_table, context_lens, page_refs, new_lens, copies, workspace, dev.sm_count,
                         static_cast<cudaStream_t>(cuda_stream));
}

pa_status pa_copy_pages(const pa_shape* shape, void* key_pages, void* value_pages, const int32_t* copies, int n,
                        void* workspace, size_t workspace_bytes, void* cuda_stream) {
    const pa_status st = check_shape(shape);
    if (st != PA_OK) return st;
    if (!on(key_pages, 16) || !on(value_pages, 16)) return PA_ERR_INVALID_ARG;
    return copy(shape, {{key_pages, value_pages, nullptr, nullptr}}, copies, n, workspace, workspace_bytes, cuda_stream);
}

pa_status pa_copy_pages_q4(const pa_shape* shape, const pa_q4_pool* pool, const int32_t* copies, int n, void* workspace,
                           size_t workspace_bytes, void* cuda_stream) {
    const pa_status st = check_shape(shape);
    if (st != PA_OK) return st;
    if (!pool_ok(pool)) return PA_ERR_INVALID_ARG;
    return copy(shape, bufs(*pool), copies, n, workspace, workspace_bytes, cuda_stream);
}

}  // extern "C"
