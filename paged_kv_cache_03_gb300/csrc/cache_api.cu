// cache_api.cu -- the extern "C" entry points of the cache operators of
// paged_attn.h: 4-bit pages, key weights and eviction.  Argument checks on the
// host, then the launches.
#include <cfloat>
#include <climits>

#include "cache.h"

namespace pa {
namespace {

bool on(const void* p, uintptr_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }

bool pool_ok(const pa_q4_pool* p) {
    return p && on(p->key_codes, 16) && on(p->value_codes, 16) && on(p->key_scales, 16) && on(p->value_scales, 16);
}

long long capacity(const pa_shape& s) { return static_cast<long long>(s.max_pages_per_seq) * s.page_size; }

pa_status device_ok(DeviceInfo* dev) {
    const pa_status st = current_device_info(dev);
    if (st != PA_OK) return st;
    return dev->cc_major == 10 && dev->cc_minor == 3 ? PA_OK : PA_ERR_UNSUPPORTED;
}

pa_status attend(const pa_shape* shape, const void* query, const void* kc, const void* vc, const void* ks,
                 const void* vs, const int32_t* bt, const int32_t* ctx, float scale, int causal,
                 const float* w_in, float* w_out, long long w_S, void* out, void* ws, size_t ws_bytes,
                 void* stream) {
    pa_status st = check_call_args(shape, query, kc, vc, bt, ctx, scale, out);
    if (st != PA_OK) return st;
    if (w_in && !w_out) return PA_ERR_INVALID_ARG;
    if (w_out && (!on(w_out, 4) || w_S < capacity(*shape) || (w_in && !on(w_in, 4)))) return PA_ERR_INVALID_ARG;
    if (!on(ws, 256)) return PA_ERR_WORKSPACE;
    WalkCall c;
    st = device_ok(&c.dev);
    if (st != PA_OK) return st;
    c.sh = *shape;
    c.q = query;
    c.kc = kc;
    c.vc = vc;
    c.ks = ks;
    c.vs = vs;
    c.bt = bt;
    c.ctx = ctx;
    c.scale = scale;
    c.causal = causal ? 1 : 0;
    c.out = out;
    c.w_in = w_in;
    c.w_out = w_out;
    c.w_S = w_out ? w_S : 0;
    c.ws = ws;
    c.ws_bytes = ws_bytes;
    c.stream = static_cast<cudaStream_t>(stream);
    return walk_launch(c);
}

pa_status evict(const pa_shape* shape, EvictCall& c, const int32_t* bt, const int32_t* ctx, const float* w,
                long long w_S, int keep, int recent, const int32_t* dst_bt, int dst_max_pages,
                int32_t* ctx_out, float* w_out, long long w_out_S, int32_t* kept, void* ws, size_t ws_bytes,
                void* stream) {
    if (!on(bt, 4) || !on(ctx, 4) || !on(w, 4) || !on(dst_bt, 4) || !on(ctx_out, 4) || !on(w_out, 4) || !on(kept, 4))
        return PA_ERR_INVALID_ARG;
    // nothing is trimmed in place
    if (ctx_out == ctx || w_out == w || dst_bt == bt) return PA_ERR_INVALID_ARG;
    if (keep < 1 || recent < 0 || recent > keep || dst_max_pages < 1) return PA_ERR_INVALID_ARG;
    if (w_S < capacity(*shape) || w_out_S < keep || static_cast<long long>(dst_max_pages) * shape->page_size < keep)
        return PA_ERR_INVALID_ARG;
    if (!on(ws, 4) || ws_bytes < kFlagBytes) return PA_ERR_WORKSPACE;
    const pa_status st = device_ok(&c.dev);
    if (st != PA_OK) return st;
    c.sh = *shape;
    c.bt = bt;
    c.ctx = ctx;
    c.w = w;
    c.w_S = w_S;
    c.keep = keep;
    c.recent = recent;
    c.dst_bt = dst_bt;
    c.dst_max_pages = dst_max_pages;
    c.ctx_out = ctx_out;
    c.w_out = w_out;
    c.w_out_S = w_out_S;
    c.kept = kept;
    c.flag = static_cast<uint32_t*>(ws);
    c.stream = static_cast<cudaStream_t>(stream);
    return evict_launch(c);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

size_t pa_q4_workspace_bytes(const pa_shape* shape, int key_weights) {
    DeviceInfo dev;
    if (check_shape(shape) != PA_OK || current_device_info(&dev) != PA_OK) return 0;
    return walk_workspace_bytes(*shape, true, key_weights != 0, dev.sm_count);
}

size_t pa_weights_workspace_bytes(const pa_shape* shape) {
    DeviceInfo dev;
    if (check_shape(shape) != PA_OK || shape->dtype != PA_BF16 || current_device_info(&dev) != PA_OK) return 0;
    return walk_workspace_bytes(*shape, false, true, dev.sm_count);
}

pa_status pa_append_kv_q4(const pa_shape* shape, const void* k_new, const void* v_new, const pa_q4_pool* pool,
                          const int32_t* block_table, const int32_t* context_lens, void* workspace,
                          size_t workspace_bytes, void* cuda_stream) {
    pa_status st = check_shape(shape);
    if (st != PA_OK) return st;
    if (!on(k_new, 16) || !on(v_new, 16) || !pool_ok(pool) || !on(block_table, 4) || !on(context_lens, 4))
        return PA_ERR_INVALID_ARG;
    if (!on(workspace, 4) || workspace_bytes < kFlagBytes) return PA_ERR_WORKSPACE;
    DeviceInfo dev;
    st = device_ok(&dev);
    if (st != PA_OK) return st;
    return q4_append_launch(*shape, k_new, v_new, *pool, block_table, context_lens,
                            static_cast<uint32_t*>(workspace), static_cast<cudaStream_t>(cuda_stream));
}

pa_status pa_gather_kv_q4(const pa_shape* shape, const pa_q4_pool* pool, const int32_t* block_table,
                          const int32_t* context_lens, int n, int tail, void* k_dense, void* v_dense,
                          void* workspace, size_t workspace_bytes, void* cuda_stream) {
    pa_status st = check_shape(shape);
    if (st != PA_OK) return st;
    if (!pool_ok(pool) || !on(block_table, 4) || !on(context_lens, 4) || !on(k_dense, 16) || !on(v_dense, 16) || n < 1)
        return PA_ERR_INVALID_ARG;
    if (!on(workspace, 4) || workspace_bytes < kFlagBytes) return PA_ERR_WORKSPACE;
    DeviceInfo dev;
    st = device_ok(&dev);
    if (st != PA_OK) return st;
    return q4_gather_launch(*shape, *pool, block_table, context_lens, n, tail ? 1 : 0, 1, nullptr, 0, k_dense, v_dense,
                            static_cast<uint32_t*>(workspace), static_cast<cudaStream_t>(cuda_stream));
}

pa_status pa_paged_attention_q4(const pa_shape* shape, const void* query, const pa_q4_pool* pool,
                                const int32_t* block_table, const int32_t* context_lens, float scale, int causal,
                                const float* key_weights, float* key_weights_out, long long weights_S, void* out,
                                void* workspace, size_t workspace_bytes, void* cuda_stream) {
    const pa_status st = check_shape(shape);
    if (st != PA_OK) return st;
    if (!pool_ok(pool)) return PA_ERR_INVALID_ARG;
    return attend(shape, query, pool->key_codes, pool->value_codes, pool->key_scales, pool->value_scales,
                  block_table, context_lens, scale, causal, key_weights, key_weights_out, weights_S, out,
                  workspace, workspace_bytes, cuda_stream);
}

pa_status pa_paged_attention_weights(const pa_shape* shape, const void* query, const void* key_pages,
                                     const void* value_pages, const int32_t* block_table,
                                     const int32_t* context_lens, float scale, int causal,
                                     const float* key_weights, float* key_weights_out, long long weights_S,
                                     void* out, void* workspace, size_t workspace_bytes, void* cuda_stream) {
    const pa_status st = check_shape(shape);
    if (st != PA_OK) return st;
    if (!key_weights_out) return PA_ERR_INVALID_ARG;
    if (shape->dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    return attend(shape, query, key_pages, value_pages, nullptr, nullptr, block_table, context_lens, scale, causal,
                  key_weights, key_weights_out, weights_S, out, workspace, workspace_bytes, cuda_stream);
}

pa_status pa_evict_kv(const pa_shape* shape, void* key_pages, void* value_pages, const int32_t* block_table,
                      const int32_t* context_lens, const float* key_weights, long long weights_S, int keep,
                      int recent, const int32_t* dst_block_table, int dst_max_pages_per_seq,
                      int32_t* context_lens_out, float* key_weights_out, long long weights_out_S, int32_t* kept,
                      void* workspace, size_t workspace_bytes, void* cuda_stream) {
    const pa_status st = check_shape(shape);
    if (st != PA_OK) return st;
    if (!on(key_pages, 16) || !on(value_pages, 16)) return PA_ERR_INVALID_ARG;
    EvictCall c = {};
    c.buf[0] = key_pages;
    c.buf[1] = value_pages;
    return evict(shape, c, block_table, context_lens, key_weights, weights_S, keep, recent, dst_block_table,
                 dst_max_pages_per_seq, context_lens_out, key_weights_out, weights_out_S, kept, workspace,
                 workspace_bytes, cuda_stream);
}

pa_status pa_evict_kv_q4(const pa_shape* shape, const pa_q4_pool* pool, const int32_t* block_table,
                         const int32_t* context_lens, const float* key_weights, long long weights_S, int keep,
                         int recent, const int32_t* dst_block_table, int dst_max_pages_per_seq,
                         int32_t* context_lens_out, float* key_weights_out, long long weights_out_S,
                         int32_t* kept, void* workspace, size_t workspace_bytes, void* cuda_stream) {
    const pa_status st = check_shape(shape);
    if (st != PA_OK) return st;
    if (!pool_ok(pool)) return PA_ERR_INVALID_ARG;
    EvictCall c = {};
    c.buf[0] = pool->key_codes;
    c.buf[1] = pool->value_codes;
    c.buf[2] = pool->key_scales;
    c.buf[3] = pool->value_scales;
    return evict(shape, c, block_table, context_lens, key_weights, weights_S, keep, recent, dst_block_table,
                 dst_max_pages_per_seq, context_lens_out, key_weights_out, weights_out_S, kept, workspace,
                 workspace_bytes, cuda_stream);
}

}  // extern "C"
