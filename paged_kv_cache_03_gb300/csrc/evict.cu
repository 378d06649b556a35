// evict.cu -- trims every (sequence, kv head) of a page pool to its heaviest
// keys: the `recent` last positions and, of the others, the keep - recent of
// the largest accumulated weight (ties: the lowest position), copied in order
// to the pages of another block table.
//
// evict_select_kernel, one CTA per (sequence, kv head): a radix select over
// the weights' bits (11, 11 and 10 of them) finds the smallest kept weight and
// how many keys of exactly that weight stay; then each warp takes a run of
// positions, and ballots and one scan over the warps give every kept position
// its place.  The keys stay in shared memory between the passes where the
// table's capacity fits.  evict_copy_kernel moves the rows: bound by HBM (each
// kept row read and written once).  Measured: 16 x 8 heads of 8192 bf16 keys halved 96 us,
// 545 MB at 5.6 TB/s, of which the selection, bound by its passes' latency, is 12; 32 x 8
// heads of 500 .. 4096 4-bit keys trimmed to 1024 about 30, the selection 13.
#include <climits>

#include "cache.h"
#include "ptx.cuh"

namespace pa {
namespace {

constexpr int kBins = 2048;
constexpr int kCached = 49152;  // keys held in shared memory (192 KB)

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

// Inclusive scan over a warp.
__device__ __forceinline__ int warp_incl(int v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

// The sum of v[0 .. n), n < 32, by a whole warp.
__device__ __forceinline__ int warp_sum_before(const int* v, int n, int lane) {
    return __reduce_add_sync(0xffffffffu, lane < n ? v[lane] : 0);
}

template <int kThreads, bool kCache>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictParams p) {
    constexpr int kWarps = kThreads / 32, kMine = kBins / kThreads;  // kMine: bins per thread
    __shared__ int hist[kBins];
    __shared__ int warp_a[kWarps], warp_b[kWarps];
    __shared__ int sel[2];
    extern __shared__ uint32_t cache[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_launch_dependents();
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
    for (int i = n + tid; i < p.keep; i += kThreads) kept[i] = -1;
    for (long long i = n + tid; i < p.w_out_S; i += kThreads) w_out[i] = 0.f;
    if (S <= p.keep) {  // all stay
        for (int i = tid; i < S; i += kThreads) {
            kept[i] = i;
            w_out[i] = w[i];
        }
        return;
    }

    const int cand = S - p.recent;  // positions that compete
    int left = p.keep - p.recent;   // of them, how many stay at or below the prefix
    uint32_t T = 0u;                // the smallest kept key
    auto key_at = [&](int i) { return kCache ? cache[i] : order_key(__ldg(w + i)); };
    for (int i = tid; i < p.recent; i += kThreads) {  // the last positions
        kept[left + i] = cand + i;
        w_out[left + i] = w[cand + i];
    }
    if (left == 0) return;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t mask = pass == 2 ? 1023u : 2047u;
#pragma unroll
        for (int k = 0; k < kMine; ++k) hist[tid + k * kThreads] = 0;
        __syncthreads();
        const int above = pass == 1 ? 21 : 10;  // bits of T already known
#pragma unroll 4
        for (int i = tid; i < cand; i += kThreads) {
            uint32_t key;
            if (kCache && pass == 0) {
                key = order_key(__ldg(w + i));
                cache[i] = key;
            } else {
                key = key_at(i);
            }
            if (pass == 0 || (key >> above) == (T >> above)) atomicAdd(&hist[(key >> shift) & mask], 1);
        }
        __syncthreads();
        // the bin that holds the left-th largest: thread tid has kMine bins, from the top
        const int top = kBins - 1 - kMine * tid;
        int c[kMine], own = 0;
#pragma unroll
        for (int k = 0; k < kMine; ++k) own += c[k] = hist[top - k];
        const int incl = warp_incl(own, lane);
        if (lane == 31) warp_a[warp] = incl;
        __syncthreads();
        int before = incl - own + warp_sum_before(warp_a, warp, lane);
        if (before < left && left <= before + own) {
#pragma unroll
            for (int k = 0; k < kMine; ++k) {
                if (before < left && left <= before + c[k]) {
                    sel[0] = top - k;
                    sel[1] = before;
                }
                before += c[k];
            }
        }
        __syncthreads();
        T |= static_cast<uint32_t>(sel[0]) << shift;
        left -= sel[1];  // (the next pass's first barrier comes before sel is written again)
    }

    // Warp v takes positions [v * run, (v + 1) * run): how many are above T, how
    // many equal; then where each kept one goes.  `left` of the equal ones stay,
    // those of the lowest positions.
    const int run = ((cand + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int i0 = warp * run, i1 = min(cand, i0 + run);
    int gt = 0, eq = 0;
#pragma unroll 4
    for (int i = i0 + lane; i - lane < i1; i += 32) {
        const uint32_t key = i < i1 ? key_at(i) : 0u;
        gt += __popc(__ballot_sync(0xffffffffu, i < i1 && key > T));
        eq += __popc(__ballot_sync(0xffffffffu, i < i1 && key == T));
    }
    if (lane == 0) {
        warp_a[warp] = gt;
        warp_b[warp] = eq;
    }
    __syncthreads();
    gt = warp_sum_before(warp_a, warp, lane);
    eq = warp_sum_before(warp_b, warp, lane);
    const uint32_t lower = (1u << lane) - 1;
#pragma unroll 4
    for (int i = i0 + lane; i - lane < i1; i += 32) {
        const uint32_t key = i < i1 ? key_at(i) : 0u;
        const float wi = i < i1 ? __ldg(w + i) : 0.f;
        const uint32_t g = __ballot_sync(0xffffffffu, i < i1 && key > T);
        const uint32_t e = __ballot_sync(0xffffffffu, i < i1 && key == T);
        const int eqb = eq + __popc(e & lower);
        if (((g >> lane) & 1u) || (((e >> lane) & 1u) && eqb < left)) {
            const int dst = gt + __popc(g & lower) + min(eqb, left);
            kept[dst] = i;
            w_out[dst] = wi;
        }
        gt += __popc(g);
        eq += __popc(e);
    }
}

struct CopyParams {
    uint8_t* buf[4];
    const int32_t* bt;
    const int32_t* dst_bt;
    const int32_t* kept;
    uint32_t* flag;
    int H_kv, keep, ps, max_npg, dst_max_npg, num_pages, ntile;
};

// A block moves ROWS kept rows of one (sequence, kv head): first their source
// and destination rows, then 16 bytes a thread and copy, four in flight.  RB:
// bytes of a K or V row; SB: bytes of its scales (4-bit pages), else 0.
template <int ROWS, int RB, int SB>
__global__ void __launch_bounds__(256) evict_copy_kernel(const CopyParams p) {
    __shared__ int src_s[ROWS], dst_s[ROWS];
    const int tile = static_cast<int>(blockIdx.x) % p.ntile, bk = static_cast<int>(blockIdx.x) / p.ntile;
    const int b = bk / p.H_kv, kvh = bk - b * p.H_kv;
    const int j0 = tile * ROWS;
    pdl_wait_primary();
    for (int i = threadIdx.x; i < ROWS; i += 256) {
        const int j = j0 + i;
        // (written by the kernel before: a plain load, which stays behind the wait)
        const int s = j < p.keep ? p.kept[static_cast<long long>(bk) * p.keep + j] : -1;
        int src = -1, dst = -1;
        if (s >= 0) {
            const int from = __ldg(p.bt + static_cast<long long>(b) * p.max_npg + s / p.ps);
            const int to = __ldg(p.dst_bt + static_cast<long long>(b) * p.dst_max_npg + j / p.ps);
            if (from >= 0 && from < p.num_pages && to >= 0 && to < p.num_pages) {
                src = (from * p.H_kv + kvh) * p.ps + s % p.ps;
                dst = (to * p.H_kv + kvh) * p.ps + j % p.ps;
            } else {
                atomicOr(p.flag, PA_FLAG_BAD_PAGE);
            }
        }
        src_s[i] = src;
        dst_s[i] = dst;
    }
    __syncthreads();
    constexpr int LPR = RB / 16, PER = ROWS * LPR / 256;  // copies per thread and buffer
    static_assert(ROWS * LPR % 256 == 0, "whole passes");
    uint4 v[2][PER];
    const int c = threadIdx.x % LPR;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int src = src_s[(threadIdx.x + 256 * i) / LPR];
            if (src >= 0)
                v[k][i] = __ldcs(reinterpret_cast<const uint4*>(p.buf[k] + static_cast<long long>(src) * RB) + c);
        }
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int dst = dst_s[(threadIdx.x + 256 * i) / LPR];
            if (dst >= 0) reinterpret_cast<uint4*>(p.buf[k] + static_cast<long long>(dst) * RB)[c] = v[k][i];
        }
    if constexpr (SB > 0) {
        static_assert(SB == 8 && ROWS == 128, "one 8-byte copy per thread: K scales, then V scales");
        const int i = threadIdx.x & 127, src = src_s[i];
        uint8_t* const buf = threadIdx.x < 128 ? p.buf[2] : p.buf[3];
        if (src >= 0)
            *reinterpret_cast<uint2*>(buf + static_cast<long long>(dst_s[i]) * SB) =
                *reinterpret_cast<const uint2*>(buf + static_cast<long long>(src) * SB);
    }
}

template <int ROWS, int RB, int SB>
pa_status launch_copy(CopyParams& q, long long bk, cudaStream_t stream) {
    q.ntile = (q.keep + ROWS - 1) / ROWS;
    if (bk * q.ntile > INT_MAX) return PA_ERR_UNSUPPORTED;
    return launch_dependent(evict_copy_kernel<ROWS, RB, SB>, dim3(static_cast<unsigned>(bk * q.ntile)), 256, 0, stream, q)
               ? PA_OK
               : PA_ERR_CUDA;
}

template <int kThreads, bool kCache>
pa_status launch_select(const EvictParams& p, long long heads, const EvictCall& c) {
    const size_t smem = kCache ? static_cast<size_t>(p.max_S) * 4 : 0;
    if (kCache) {
        static int attr_done[64] = {0};
        if (!attr_done[c.dev.device]) {
            if (cudaFuncSetAttribute(evict_select_kernel<kThreads, kCache>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kCached * 4) != cudaSuccess)
                return PA_ERR_CUDA;
            attr_done[c.dev.device] = 1;
        }
    }
    evict_select_kernel<kThreads, kCache><<<static_cast<unsigned>(heads), kThreads, smem, c.stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

pa_status evict_launch(const EvictCall& c) {
    const pa_shape& sh = c.sh;
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
    const long long bk = static_cast<long long>(sh.B) * sh.H_kv;
    if (bk * ((c.keep + 15ll) / 16) > INT_MAX) return PA_ERR_UNSUPPORTED;
    // 1024 threads, or 512 where the heads are more than are resident with 1024 (1024,
    // 512, us for select and copy and read-back: 512 heads of 4096 keys 77, 73, of
    // about 1000 62, 59; 64 heads of 4096 24, 26; 16 of 32768 54, 73).
    pa_status st;
    if (p.max_S > kCached)
        st = launch_select<1024, false>(p, bk, c);
    else if (bk > 2ll * c.dev.sm_count)
        st = launch_select<512, true>(p, bk, c);
    else
        st = launch_select<1024, true>(p, bk, c);
    if (st != PA_OK) return st;
    CopyParams q;
    for (int k = 0; k < 4; ++k) q.buf[k] = static_cast<uint8_t*>(c.buf[k]);
    q.bt = c.bt;
    q.dst_bt = c.dst_bt;
    q.kept = c.kept;
    q.flag = c.flag;
    q.H_kv = sh.H_kv;
    q.keep = c.keep;
    q.ps = sh.page_size;
    q.max_npg = sh.max_pages_per_seq;
    q.dst_max_npg = c.dst_max_pages;
    q.num_pages = sh.num_pages;
    if (c.buf[2]) return launch_copy<128, kQ4CodeBytes, kQ4Groups>(q, bk, c.stream);
    return sh.dtype == PA_BF16 ? launch_copy<32, 2 * kHeadDim, 0>(q, bk, c.stream)
                               : launch_copy<16, 4 * kHeadDim, 0>(q, bk, c.stream);
}

}  // namespace pa
