// tree.cu -- which drafts a draft sees, and the accepted drafts' rows moved together.
//
// The drafts of a sequence are its last L positions; parents[i] < i is the draft that
// draft i follows, -1 the last position before the drafts, -2 no draft.
#include <climits>

#include "tree.h"
#include "ptx.cuh"

namespace pa {
namespace {

// ---- visibility -------------------------------------------------------------------
// mask[i] = {i} + mask[parents[i]], as bits; no draft, or a draft after none: 0.
//
// One CTA per sequence, warp k drafts 32 k .. 32 k + 31.  A parent comes before its
// children, so within a warp five rounds of pointer doubling by shuffles give every draft
// its ancestors in the warp, one word, and the one before them (`up`); then every draft
// follows the `up`s, at most one a warp before its own, and takes their words.  A chain of
// latencies: 64 trees of 64 drafts 2.2 us, 8 of 1001 drafts 7 us (14 when all warps took 32
// drafts after 32 with a barrier for each).
__global__ void __launch_bounds__(1024) tree_mask_kernel(const int32_t* parents, uint32_t* mask, int32_t* depths,
                                                         uint32_t* flag, int L, int W) {
    extern __shared__ uint32_t rows[];  // [32 W][W | 1], then [32 W] of word and `up`
    const int stride = W | 1;           // odd: a word of 32 rows lies in 32 banks
    int2* const drafts = reinterpret_cast<int2*>(rows + 32 * W * stride);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long first = static_cast<long long>(blockIdx.x) * L;
    const int parent = tid < L ? __ldg(parents + first + tid) : -2;
    bool lost = parent < -1 || parent >= tid;
    if (tid < L && (parent < -2 || parent >= tid)) atomicOr(flag, PA_FLAG_BAD_TREE);
    int anc = lost || parent < 32 * warp ? -1 : parent & 31;  // lane of an ancestor
    int up = lost || anc >= 0 ? -1 : parent;                  // ancestor before this warp, -1: none
    uint32_t bits = 1u << lane;
#pragma unroll
    for (int r = 0; r < 5; ++r) {
        const int from = anc < 0 ? lane : anc;
        const uint32_t b = __shfl_sync(0xffffffffu, bits, from);
        const int u = __shfl_sync(0xffffffffu, up, from), a = __shfl_sync(0xffffffffu, anc, from);
        const bool l = __shfl_sync(0xffffffffu, static_cast<int>(lost), from);
        if (anc >= 0) {
            bits |= b;
            up = u;
            lost |= l;
            anc = a;
        }
    }
    uint32_t* const mine = rows + tid * stride;
    if (warp < W) {
        drafts[tid] = lost ? make_int2(0, -1) : make_int2(static_cast<int>(bits), up);
        for (int w = 0; w < W; ++w) mine[w] = w == warp && !lost ? bits : 0u;
    }
    __syncthreads();
    if (tid < L) {
        int depth = __popc(bits) - 1;
        if (!lost)
            for (int u = up; u >= 0;) {
                const int2 d = drafts[u];
                if (d.x == 0) {  // no draft, so this one is none
                    lost = true;
                    break;
                }
                mine[u >> 5] = static_cast<uint32_t>(d.x);
                depth += __popc(d.x);
                u = d.y;
            }
        if (lost)
            for (int w = 0; w < W; ++w) mine[w] = 0u;
        depths[first + tid] = lost ? -1 : depth;
    }
    __syncthreads();
    const int warps = static_cast<int>(blockDim.x) >> 5;
    // 2^shift lanes a row
    const int shift = W > 1 ? 32 - __clz(W - 1) : 0, per = 32 >> shift, w = lane & ((1 << shift) - 1);
#pragma unroll 4
    for (int r = warp * per + (lane >> shift); r < L; r += warps * per)
        if (w < W) mask[(first + r) * W + w] = rows[r * stride + w];
}

// ---- compaction -------------------------------------------------------------------
struct CompactParams {
    uint8_t* buf[4];
    int row_bytes[4];
    const int32_t* bt;
    const int32_t* ctx;
    const int32_t* path;
    const int32_t* path_lens;
    int32_t* ctx_out;
    uint32_t* flag;
    int H_kv, L, path_n, ps, max_npg, num_pages;
    long long max_S;
};

// Row path[j] of the drafts to place j of a (sequence, kv head) in one buffer.  The path
// ascends, so path[j] >= j: the rows of a pass are read before any is written, and later
// passes read behind what earlier ones wrote.  U: 16 bytes, or 8 (scales of a row).
template <class U>
__device__ __forceinline__ void compact_rows(const CompactParams& p, uint8_t* buf, int row_bytes, int b, int kvh, int first,
                                             int n, bool& bad_page) {
    const int units = row_bytes / static_cast<int>(sizeof(U)), per = static_cast<int>(blockDim.x) / units;
    const int c = static_cast<int>(threadIdx.x) % units, at = static_cast<int>(threadIdx.x) / units;
    const int32_t* const path = p.path + static_cast<long long>(b) * p.path_n;
    auto row = [&](int s) -> U* {
        const int page = __ldg(p.bt + static_cast<long long>(b) * p.max_npg + s / p.ps);
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) {
            bad_page = true;
            return nullptr;
        }
        return reinterpret_cast<U*>(buf + ((static_cast<long long>(page) * p.H_kv + kvh) * p.ps + s % p.ps) * row_bytes) + c;
    };
    for (int j0 = 0; j0 < n; j0 += per) {
        const int j = j0 + at;
        U* to = nullptr;
        U v;
        if (j < n) {
            const int i = __ldg(path + j);
            if (i != j) {
                to = row(first + j);
                const U* const from = row(first + i);
                if (from)
                    v = *from;
                else
                    to = nullptr;
            }
        }
        __syncthreads();
        if (to) *to = v;
    }
}

// A CTA per (sequence, kv head) and buffer.  Few rows: what it takes is its chain of
// dependent loads (path, page, row), 6 to 9 us for 64 sequences.
__global__ void __launch_bounds__(256) compact_kernel(const CompactParams p) {
    const int b = static_cast<int>(blockIdx.x) / p.H_kv, kvh = static_cast<int>(blockIdx.x) - b * p.H_kv;
    const bool writes = threadIdx.x == 0 && kvh == 0 && blockIdx.y == 0;  // lengths and flags
    const int S = __ldg(p.ctx + b), n = __ldg(p.path_lens + b);
    const int32_t* const path = p.path + static_cast<long long>(b) * p.path_n;
    // (the first entries are requested beside their number)
    const int early = threadIdx.x < p.path_n ? __ldg(path + threadIdx.x) : 0;
    if (S < p.L || static_cast<long long>(S) > p.max_S) {
        if (writes) {
            p.ctx_out[b] = S;
            atomicOr(p.flag, PA_FLAG_BAD_CONTEXT);
        }
        return;
    }
    bool bad = n < 0 || n > p.L || n > p.path_n;
    if (!bad)
        for (int j = threadIdx.x; j < n; j += blockDim.x) {
            const int i = j == threadIdx.x ? early : __ldg(path + j), before = j > 0 ? __ldg(path + j - 1) : -1;
            bad |= i <= before || i >= p.L;
        }
    bad = __syncthreads_or(bad);
    const int first = S - p.L;
    if (writes) {
        p.ctx_out[b] = bad ? first : first + n;
        if (bad) atomicOr(p.flag, PA_FLAG_BAD_TREE);
    }
    if (bad) return;
    bool bad_page = false;
    const int rb = p.row_bytes[blockIdx.y];
    if (rb >= 16)
        compact_rows<uint4>(p, p.buf[blockIdx.y], rb, b, kvh, first, n, bad_page);
    else
        compact_rows<uint2>(p, p.buf[blockIdx.y], rb, b, kvh, first, n, bad_page);
    if (bad_page) atomicOr(p.flag, PA_FLAG_BAD_PAGE);
}

}  // namespace

pa_status tree_mask_launch(int B, int L, const int32_t* parents, uint32_t* mask, int32_t* depths, uint32_t* flag,
                           cudaStream_t stream) {
    const int W = tree_words(L);
    const size_t smem = (32ull * W * (W | 1) + 64ull * W) * 4;
    static int attr_done[64] = {0};
    DeviceInfo dev;
    const pa_status st = current_device_info(&dev);
    if (st != PA_OK) return st;
    if (!attr_done[dev.device]) {
        constexpr int most = (kTreeMax * (kTreeMax / 32 + 1) + 2 * kTreeMax) * 4;
        if (cudaFuncSetAttribute(tree_mask_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
            return PA_ERR_CUDA;
        attr_done[dev.device] = 1;
    }
    const int threads = W > 8 ? 32 * W : 256;  // (small trees: more warps for the writes)
    tree_mask_kernel<<<static_cast<unsigned>(B), static_cast<unsigned>(threads), smem, stream>>>(parents, mask, depths,
                                                                                                 flag, L, W);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status compact_launch(const CompactCall& c) {
    const pa_shape& sh = c.sh;
    const long long heads = static_cast<long long>(sh.B) * sh.H_kv;
    if (heads > INT_MAX) return PA_ERR_UNSUPPORTED;
    CompactParams p;
    const bool q4 = c.pool.buf[2] != nullptr;
    for (int k = 0; k < 4; ++k) {
        p.buf[k] = static_cast<uint8_t*>(c.pool.buf[k]);
        p.row_bytes[k] = q4 ? (k < 2 ? kQ4CodeBytes : kQ4Groups) : (sh.dtype == PA_BF16 ? 2 : 4) * kHeadDim;
    }
    p.bt = c.bt;
    p.ctx = c.ctx;
    p.path = c.path;
    p.path_lens = c.path_lens;
    p.ctx_out = c.ctx_out;
    p.flag = c.flag;
    p.H_kv = sh.H_kv;
    p.L = sh.L;
    p.path_n = c.path_n;
    p.ps = sh.page_size;
    p.max_npg = sh.max_pages_per_seq;
    p.num_pages = sh.num_pages;
    p.max_S = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    compact_kernel<<<dim3(static_cast<unsigned>(heads), q4 ? 4 : 2), 256, 0, c.stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
