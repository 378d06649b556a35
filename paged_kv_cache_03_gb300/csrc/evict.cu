// evict.cu -- trims every (sequence, kv head) of a page pool to its heaviest
// keys: the `recent` last positions and, of the others, the keep - recent of
// the largest accumulated weight (ties: the lowest position), copied in order
// to the pages of another block table.
//
// evict_select_kernel, one CTA per (sequence, kv head): a radix select over
// the weights' bits finds the smallest kept weight and how many keys of
// exactly that weight stay; a block scan in position order then writes the
// kept positions and their weights.  evict_copy_kernel moves the rows.
#include <climits>

#include "cache.h"

namespace pa {
namespace {

constexpr int kThreads = 512;

struct EvictParams {
    const int32_t* bt;
    const int32_t* ctx;
    const float* w;
    long long w_S;
    int keep, recent;
    int32_t* ctx_out;
    float* w_out;
    long long w_out_S;
    int32_t* kept;
    uint32_t* flag;
    int H_kv;
    long long max_S;
};

// Unsigned key in the order of the weights; +-0 are one value, NaN is above all.
__device__ __forceinline__ uint32_t order_key(float w) {
    if (w != w) return 0xffffffffu;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = +0
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictParams p) {
    __shared__ int hist[256];
    __shared__ int warp_sum[kThreads / 32];
    __shared__ int sel[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = static_cast<int>(blockIdx.x) / p.H_kv, kvh = static_cast<int>(blockIdx.x) % p.H_kv;
    int S = __ldg(p.ctx + b);
    if (S < 0 || static_cast<long long>(S) > p.max_S) {
        if (tid == 0 && kvh == 0) atomicOr(p.flag, PA_FLAG_BAD_CONTEXT);
        S = 0;
    }
    const float* const w = p.w + static_cast<long long>(blockIdx.x) * p.w_S;
    int32_t* const kept = p.kept + static_cast<long long>(blockIdx.x) * p.keep;
    float* const w_out = p.w_out + static_cast<long long>(blockIdx.x) * p.w_out_S;
    const int n = min(S, p.keep);
    if (tid == 0 && kvh == 0) p.ctx_out[b] = n;

    const bool all = S <= p.keep;
    const int cand = all ? 0 : S - p.recent;  // positions that compete
    uint32_t T = 0u;                          // the smallest kept key
    int left = all ? 0 : p.keep - p.recent;   // keys still to find at or below the prefix
    if (!all && left > 0) {
#pragma unroll 1
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int base = 0; base < cand; base += kThreads) {
                const int i = base + tid;
                const uint32_t key = i < cand ? order_key(w[i]) : 0u;
                const bool in = i < cand && (shift == 24 || (key >> (shift + 8)) == (T >> (shift + 8)));
                const uint32_t bin = in ? (key >> shift) & 255u : 256u;
                const uint32_t same = __match_any_sync(0xffffffffu, bin);
                if (in && lane == __ffs(same) - 1) atomicAdd(&hist[bin], __popc(same));
            }
            __syncthreads();
            if (tid == 0) {
                int c = 0, v = 255;
                while (v > 0 && c + hist[v] < left) c += hist[v--];
                sel[0] = v;
                sel[1] = c;
            }
            __syncthreads();
            T |= static_cast<uint32_t>(sel[0]) << shift;
            left -= sel[1];
            __syncthreads();
        }
    }
    // `left` keys equal to T stay, those of the lowest positions
    int gt_before = 0, eq_before = 0;  // over earlier positions
    for (int base = 0; base < S; base += kThreads) {
        const int i = base + tid;
        const float wi = i < S ? w[i] : 0.f;
        const uint32_t key = order_key(wi);
        const bool fixed = i < S && (all || i >= cand);
        const bool gt = fixed || (i < cand && p.keep > p.recent && key > T);
        const bool eq = !fixed && i < cand && p.keep > p.recent && key == T;
        // counts of both kinds up to and including this thread, packed
        int x = (gt ? 1 : 0) | (eq ? 1 << 16 : 0);
        const int own = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) warp_sum[warp] = x;
        __syncthreads();
        int before = x - own, total = 0;
#pragma unroll
        for (int v = 0; v < kThreads / 32; ++v) {
            const int y = warp_sum[v];
            if (v < warp) before += y;
            total += y;
        }
        __syncthreads();
        const int eqb = eq_before + (before >> 16), gtb = gt_before + (before & 0xffff);
        if (gt || (eq && eqb < left)) {
            const int dst = gtb + min(eqb, left);
            kept[dst] = i;
            w_out[dst] = wi;
        }
        gt_before += total & 0xffff;
        eq_before += total >> 16;
    }
    for (int i = n + tid; i < p.keep; i += kThreads) kept[i] = -1;
    for (long long i = n + tid; i < p.w_out_S; i += kThreads) w_out[i] = 0.f;
}

struct CopyParams {
    uint8_t* buf[4];
    int row_bytes[4];
    int nbuf;
    const int32_t* bt;
    const int32_t* dst_bt;
    const int32_t* kept;
    uint32_t* flag;
    long long rows;  // B * H_kv * keep
    int H_kv, keep, ps, max_npg, dst_max_npg, num_pages;
};

// One warp per kept row.
__global__ void __launch_bounds__(256) evict_copy_kernel(const CopyParams p) {
    const int lane = threadIdx.x & 31;
    for (long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); row < p.rows;
         row += static_cast<long long>(gridDim.x) * 8) {
        const int s = p.kept[row];
        if (s < 0) continue;
        const long long bk = row / p.keep;
        const int j = static_cast<int>(row - bk * p.keep);
        const int b = static_cast<int>(bk / p.H_kv);
        const int kvh = static_cast<int>(bk - static_cast<long long>(b) * p.H_kv);
        const int from = __ldg(p.bt + static_cast<long long>(b) * p.max_npg + s / p.ps);
        const int to = __ldg(p.dst_bt + static_cast<long long>(b) * p.dst_max_npg + j / p.ps);
        if (from < 0 || from >= p.num_pages || to < 0 || to >= p.num_pages) {
            if (lane == 0) atomicOr(p.flag, PA_FLAG_BAD_PAGE);
            continue;
        }
        const long long src = (static_cast<long long>(from) * p.H_kv + kvh) * p.ps + s % p.ps;
        const long long dst = (static_cast<long long>(to) * p.H_kv + kvh) * p.ps + j % p.ps;
        for (int k = 0; k < p.nbuf; ++k)
            for (int o = 8 * lane; o < p.row_bytes[k]; o += 256)
                *reinterpret_cast<uint2*>(p.buf[k] + dst * p.row_bytes[k] + o) =
                    *reinterpret_cast<const uint2*>(p.buf[k] + src * p.row_bytes[k] + o);
    }
}

}  // namespace

pa_status evict_launch(const EvictCall& c) {
    const pa_shape& sh = c.sh;
    if (static_cast<long long>(sh.B) * sh.H_kv > INT_MAX) return PA_ERR_UNSUPPORTED;
    EvictParams p;
    p.bt = c.bt;
    p.ctx = c.ctx;
    p.w = c.w;
    p.w_S = c.w_S;
    p.keep = c.keep;
    p.recent = c.recent;
    p.ctx_out = c.ctx_out;
    p.w_out = c.w_out;
    p.w_out_S = c.w_out_S;
    p.kept = c.kept;
    p.flag = c.flag;
    p.H_kv = sh.H_kv;
    p.max_S = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    evict_select_kernel<<<static_cast<unsigned>(sh.B * sh.H_kv), kThreads, 0, c.stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
    CopyParams q;
    for (int k = 0; k < 4; ++k) {
        q.buf[k] = static_cast<uint8_t*>(c.buf[k]);
        q.row_bytes[k] = c.row_bytes[k];
    }
    q.nbuf = c.nbuf;
    q.bt = c.bt;
    q.dst_bt = c.dst_bt;
    q.kept = c.kept;
    q.flag = c.flag;
    q.rows = static_cast<long long>(sh.B) * sh.H_kv * c.keep;
    q.H_kv = sh.H_kv;
    q.keep = c.keep;
    q.ps = sh.page_size;
    q.max_npg = sh.max_pages_per_seq;
    q.dst_max_npg = c.dst_max_pages;
    q.num_pages = sh.num_pages;
    const long long blocks = (q.rows + 7) / 8, cap = 8ll * c.dev.sm_count;
    evict_copy_kernel<<<static_cast<unsigned>(blocks < cap ? blocks : cap), 256, 0, c.stream>>>(q);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
