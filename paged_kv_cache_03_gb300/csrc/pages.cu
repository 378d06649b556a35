// pages.cu -- pages shared between sequences: forking, growing, shrinking and
// freeing block-table rows with a count of holders per page, and copying the rows
// of a page that a sequence is about to write to while others hold it.
//
// refs[p] is the number of block-table rows that name page p; 0 is a free page.
//   fork    rows of a table named twice: refs + 1 for every page.
//   resize  shorter: refs - 1 for the pages past the new end; longer: the lowest free
//           pages, and a page of its own in the place of a partly filled last page
//           that others hold (its rows are to be copied: `copies`).
// Everything is decided by sequence and page number, never by the order of atomics, so
// equal calls give equal tables.
#include <climits>

#include "tree.h"
#include "ptx.cuh"

namespace pa {
namespace {

struct PagesParams {
    int32_t* bt;
    int32_t* ctx;
    int32_t* refs;
    uint32_t* flag;
    int B, num_pages, ps, max_npg;
    long long max_S;
    __device__ __forceinline__ int pages(int len) const { return (len + ps - 1) / ps; }
    __device__ __forceinline__ bool len_ok(int len) const { return len >= 0 && static_cast<long long>(len) <= max_S; }
    __device__ __forceinline__ bool page_ok(int p) const {
        return static_cast<unsigned>(p) < static_cast<unsigned>(num_pages);
    }
    __device__ __forceinline__ int32_t* row(int b) const { return bt + static_cast<long long>(b) * max_npg; }
};

// ---- fork -------------------------------------------------------------------------
// One CTA per fork.  What a CTA reads of the table and the lengths no other writes: of the
// forks that name a target the first alone may have it, and a fork whose source any fork names
// as its target is refused, whether or not that one is made (which another CTA decides).
// Bound by the atomics of shared pages: 64 forks of up to 32 pages 4 us, 48 of up to 2000
// pages 7.
__global__ void __launch_bounds__(256) fork_kernel(const PagesParams p, const int32_t* sources, const int32_t* targets,
                                                   const int32_t* lens, int n) {
    const int f = blockIdx.x, tid = threadIdx.x;
    const int src = __ldg(sources + f), tgt = __ldg(targets + f);
    bool bad = static_cast<unsigned>(src) >= static_cast<unsigned>(p.B) ||
               static_cast<unsigned>(tgt) >= static_cast<unsigned>(p.B);
    for (int i = tid; i < n; i += 256) {
        const int t = __ldg(targets + i);
        bad |= t == src || (i < f && t == tgt);
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) atomicOr(p.flag, PA_FLAG_BAD_CONTEXT);
        return;
    }
    const int S = p.ctx[src], len = lens ? __ldg(lens + f) : S;
    if (!p.len_ok(S) || len < 0 || len > S || p.ctx[tgt] != 0) {
        if (tid == 0) atomicOr(p.flag, PA_FLAG_BAD_CONTEXT);
        return;
    }
    const int32_t* const from = p.row(src);
    int32_t* const to = p.row(tgt);
    const int end = p.pages(len);
    bool bad_page = false;
    for (int e = tid; e < p.max_npg; e += 256) {
        const int page = e < end ? from[e] : -1;
        to[e] = page;
        if (e < end) {
            if (p.page_ok(page))
                atomicAdd(p.refs + page, 1);
            else
                bad_page = true;
        }
    }
    if (bad_page) atomicOr(p.flag, PA_FLAG_BAD_PAGE);
    __syncthreads();  // every thread has seen the target's old length
    if (tid == 0) p.ctx[tgt] = len;
}

// ---- resize -----------------------------------------------------------------------
struct ResizeParams {
    PagesParams t;
    const int32_t* new_lens;
    int32_t* copies;  // [B, 3] source page, new page, rows
    int* done;        // CTAs that are through with the first part
    int* list;        // free pages, ascending
    int2* share;      // per page: sequences that grow from it, the last of them
    int2* need;       // per sequence: pages taken before it, what it takes
    int chunks;       // of 32 table entries per sequence
};

constexpr int kKeeps = 1 << 30, kCopies = 1 << 29, kTakes = kCopies - 1;  // bits of need.y

// A sequence that grows: its lengths, and the partly filled last page where others hold it
// too (-1: none), with its holders.
struct Growth {
    int S, n, page, refs;
    bool grows;
};

// All CTAs give back the pages past new ends; the last one to finish then finds the free
// pages and hands them out, so growing sequences can have what shrinking ones gave up.
// Releasing is bound by the rate of atomics and spreads over the SMs; handing out is a
// chain of short steps on one SM, each a round trip to L2: what a sequence is about to do is
// read once where a thread has one sequence, and the first counts are read ahead.  80
// rows 9 to 11 us, where 64 end and where 64 grow.
__global__ void __launch_bounds__(1024) resize_kernel(const ResizeParams p) {
    const PagesParams& t = p.t;
    __shared__ int sums[32];
    __shared__ int last_cta, found;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t flags = 0u;
    const long long items = static_cast<long long>(t.B) * p.chunks;
    for (long long item = 32ll * blockIdx.x + warp; item < items; item += 32ll * gridDim.x) {
        const int b = static_cast<int>(item / p.chunks);
        const int e = static_cast<int>(item - static_cast<long long>(b) * p.chunks) * 32 + lane;
        const int S = t.ctx[b], n = __ldg(p.new_lens + b);
        if (n < 0 || n >= S || !t.len_ok(S) || e < t.pages(n) || e >= t.pages(S)) continue;
        const int page = t.row(b)[e];
        t.row(b)[e] = -1;
        if (!t.page_ok(page)) {
            flags |= PA_FLAG_BAD_PAGE;
        } else if (atomicSub(t.refs + page, 1) <= 0) {  // nobody held it: as it was
            atomicAdd(t.refs + page, 1);
            flags |= PA_FLAG_BAD_PAGE;
        }
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) last_cta = atomicAdd(p.done, 1) == static_cast<int>(gridDim.x) - 1;
    __syncthreads();
    if (flags) atomicOr(t.flag, flags);
    if (!last_cta) return;
    __threadfence();
    flags = 0u;
    if (tid == 0) {
        *p.done = 0;
        found = 0;
    }

    // the first free pages, and this thread's first sequence
    uint32_t is_free[8];
    auto look = [&](int p0) {  // a warp takes 256 counts
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int page = p0 + 256 * warp + 32 * k + lane;
            is_free[k] = page < t.num_pages && __ldcg(t.refs + page) == 0 ? 1u : 0u;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) is_free[k] = __ballot_sync(0xffffffffu, is_free[k] != 0u);
    };
    auto growth = [&](int b) {
        Growth g;
        g.S = t.ctx[b];
        g.n = __ldg(p.new_lens + b);
        g.grows = g.n > g.S && t.len_ok(g.S) && t.len_ok(g.n);
        g.page = -1;
        g.refs = 0;
        if (g.grows && g.S % t.ps != 0) {
            const int page = t.row(b)[g.S / t.ps];
            if (t.page_ok(page)) {
                g.refs = __ldcg(t.refs + page);
                if (g.refs > 1) g.page = page;
            }
        }
        return g;
    };
    Growth mine = {};
    if (tid < t.B) mine = growth(tid);
    look(0);
    auto growth_of = [&](int b) { return b == tid ? mine : growth(b); };
    for (int b = tid; b < t.B; b += 1024) {
        const Growth g = growth_of(b);
        if (g.page >= 0) p.share[g.page] = make_int2(0, -1);
    }
    __syncthreads();
    for (int b = tid; b < t.B; b += 1024) {
        const Growth g = growth_of(b);
        if (g.page < 0) continue;
        atomicAdd(&p.share[g.page].x, 1);
        atomicMax(&p.share[g.page].y, b);
    }
    __syncthreads();
    // what every sequence takes, and what those before it take
    int total = 0;
    for (int b0 = 0; b0 < t.B; b0 += 1024) {
        const int b = b0 + tid;
        int take = 0, bits = 0;
        if (b < t.B) {
            const Growth g = growth_of(b);
            if (g.grows) {
                take = t.pages(g.n) - t.pages(g.S);
                if (g.page >= 0) {
                    // where all its holders grow, the last of them keeps it
                    const int2 s = __ldcg(&p.share[g.page]);
                    if (s.x == g.refs && s.y == b) {
                        bits = kKeeps;
                    } else {
                        bits = kCopies;
                        ++take;
                    }
                }
            }
        }
        int incl = take;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        const int before = __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane] : 0);
        const int all = __reduce_add_sync(0xffffffffu, sums[lane]);
        if (b < t.B) p.need[b] = make_int2(total + before + incl - take, take | bits);
        total += all;
        __syncthreads();
    }
    // the lowest free pages (unsigned: the step behind the last pages may pass 2^31)
    for (uint32_t next = 0; next < static_cast<uint32_t>(t.num_pages) && total > 0; next += 8192) {
        const int p0 = static_cast<int>(next);
        if (p0 > 0) look(p0);
        int free_here = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) free_here += __popc(is_free[k]);
        if (lane == 0) sums[warp] = free_here;
        __syncthreads();
        int at = found + __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane] : 0);
        const int all = __reduce_add_sync(0xffffffffu, sums[lane]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = at + __popc(is_free[k] & ((1u << lane) - 1u));
            if ((is_free[k] >> lane & 1u) && i < total) p.list[i] = p0 + 256 * warp + 32 * k + lane;
            at += __popc(is_free[k]);
        }
        __syncthreads();
        if (tid == 0) found += all;
        __syncthreads();
        if (found >= total) break;
    }
    const int have = min(found, total);
    // hand them out, a warp per sequence
    for (int b = warp; b < t.B; b += 32) {
        const int S = t.ctx[b], n = __ldg(p.new_lens + b);
        const int2 need = p.need[b];
        int32_t copy[3] = {-1, -1, 0};
        if (n > S && t.len_ok(S) && t.len_ok(n)) {
            const int take = need.y & kTakes;
            // (a page is kept only where every other holder had one for its copy)
            if ((take > 0 || (need.y & kKeeps)) && static_cast<long long>(need.x) + take > have) {
                flags |= PA_FLAG_NO_PAGES;
            } else {
                const int first = need.y & kCopies ? S / t.ps : t.pages(S);  // the entry of the first new page
                if (need.y & kCopies) {
                    copy[0] = t.row(b)[first];
                    copy[1] = p.list[need.x];
                    copy[2] = S % t.ps;
                    if (lane == 0) atomicSub(t.refs + copy[0], 1);
                }
                __syncwarp();
                for (int k = lane; k < take; k += 32) {
                    const int page = p.list[need.x + k];
                    t.refs[page] = 1;
                    t.row(b)[first + k] = page;
                }
                __syncwarp();
                if (lane == 0) t.ctx[b] = n;
            }
        } else if (n >= 0) {
            if (!t.len_ok(S) || !t.len_ok(n))
                flags |= PA_FLAG_BAD_CONTEXT;
            else if (lane == 0)
                t.ctx[b] = n;  // (not longer)
        }
        if (lane < 3) p.copies[3ll * b + lane] = copy[lane];
    }
    if (flags && lane == 0) atomicOr(t.flag, flags);
}

// ---- copies -----------------------------------------------------------------------
struct CopyParams {
    uint8_t* buf[4];
    int row_bytes[4];
    const int32_t* copies;
    uint32_t* flag;
    int H_kv, num_pages, ps;
};

template <class U>
__device__ __forceinline__ void copy_units(U* dst, const U* src, long long n) {
    for (long long i = threadIdx.x; i < n; i += 4 * 256) {
        U v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + 256 * k < n) v[k] = __ldcs(src + i + 256 * k);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + 256 * k < n) dst[i + 256 * k] = v[k];
    }
}

// A CTA per (copy, kv head) and buffer: the first rows of one page to another, one
// contiguous run of bytes.  Bound by latency, a launch, the copy's entry and two rounds of
// loads a thread: 64 copies of up to 128 rows of 8 heads in bf16 9 us, of whose 16 MB HBM would
// take 3.
__global__ void __launch_bounds__(256) copy_pages_kernel(const CopyParams p) {
    const int i = static_cast<int>(blockIdx.x) / p.H_kv, h = static_cast<int>(blockIdx.x) - i * p.H_kv;
    const int src = p.copies[3ll * i], dst = p.copies[3ll * i + 1], rows = p.copies[3ll * i + 2];
    if (dst == -1 || rows == 0) return;  // none
    if (static_cast<unsigned>(src) >= static_cast<unsigned>(p.num_pages) ||
        static_cast<unsigned>(dst) >= static_cast<unsigned>(p.num_pages) ||
        static_cast<unsigned>(rows) > static_cast<unsigned>(p.ps)) {
        if (threadIdx.x == 0) atomicOr(p.flag, PA_FLAG_BAD_PAGE);
        return;
    }
    if (src == dst) return;
    const int rb = p.row_bytes[blockIdx.y];
    uint8_t* const buf = p.buf[blockIdx.y];
    const long long page = static_cast<long long>(p.ps) * rb;
    const uint8_t* const from = buf + (static_cast<long long>(src) * p.H_kv + h) * page;
    uint8_t* const to = buf + (static_cast<long long>(dst) * p.H_kv + h) * page;
    const long long n = static_cast<long long>(rows) * rb;
    if (rb >= 16)
        copy_units(reinterpret_cast<uint4*>(to), reinterpret_cast<const uint4*>(from), n / 16);
    else  // 8 bytes of scales a row: pages of odd sizes start on 8 bytes
        copy_units(reinterpret_cast<uint2*>(to), reinterpret_cast<const uint2*>(from), n / 8);
}

PagesParams pages_params(const pa_shape& sh, int32_t* bt, int32_t* ctx, int32_t* refs, uint32_t* flag) {
    PagesParams p;
    p.bt = bt;
    p.ctx = ctx;
    p.refs = refs;
    p.flag = flag;
    p.B = sh.B;
    p.num_pages = sh.num_pages;
    p.ps = sh.page_size;
    p.max_npg = sh.max_pages_per_seq;
    p.max_S = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    return p;
}

}  // namespace

pa_status fork_launch(const pa_shape& sh, int32_t* bt, int32_t* ctx, int32_t* refs, const int32_t* sources,
                      const int32_t* targets, const int32_t* lens, int n, uint32_t* flag, cudaStream_t stream) {
    fork_kernel<<<static_cast<unsigned>(n), 256, 0, stream>>>(pages_params(sh, bt, ctx, refs, flag), sources, targets,
                                                              lens, n);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

size_t pages_workspace_bytes(const pa_shape& sh) {
    return kFlagBytes + align_up(4 * static_cast<size_t>(sh.num_pages), 256) +
           align_up(8 * static_cast<size_t>(sh.num_pages), 256) + align_up(8 * static_cast<size_t>(sh.B), 256);
}

pa_status resize_launch(const pa_shape& sh, int32_t* bt, int32_t* ctx, int32_t* refs, const int32_t* new_lens,
                        int32_t* copies, void* ws, int sm_count, cudaStream_t stream) {
    // the pages that all sequences take are counted in bits below kCopies
    if (static_cast<long long>(sh.B) * (sh.max_pages_per_seq + 1ll) >= kTakes) return PA_ERR_UNSUPPORTED;
    uint8_t* const w = static_cast<uint8_t*>(ws);
    ResizeParams p;
    p.t = pages_params(sh, bt, ctx, refs, static_cast<uint32_t*>(ws));
    p.new_lens = new_lens;
    p.copies = copies;
    p.done = reinterpret_cast<int*>(w + kPagesCounterOffset);
    size_t off = kFlagBytes;
    p.list = reinterpret_cast<int*>(w + off);
    off += align_up(4 * static_cast<size_t>(sh.num_pages), 256);
    p.share = reinterpret_cast<int2*>(w + off);
    off += align_up(8 * static_cast<size_t>(sh.num_pages), 256);
    p.need = reinterpret_cast<int2*>(w + off);
    p.chunks = (sh.max_pages_per_seq + 31) / 32;
    const long long ctas = (static_cast<long long>(sh.B) * p.chunks + 31) / 32, most = 2ll * sm_count;
    resize_kernel<<<static_cast<unsigned>(ctas < most ? ctas : most), 1024, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status copy_pages_launch(const pa_shape& sh, const PoolBufs& pool, const int32_t* copies, int n, uint32_t* flag,
                            cudaStream_t stream) {
    if (static_cast<long long>(n) * sh.H_kv > INT_MAX) return PA_ERR_UNSUPPORTED;
    CopyParams p;
    const bool q4 = pool.buf[2] != nullptr;
    for (int k = 0; k < 4; ++k) {
        p.buf[k] = static_cast<uint8_t*>(pool.buf[k]);
        p.row_bytes[k] = q4 ? (k < 2 ? kQ4CodeBytes : kQ4Groups) : (sh.dtype == PA_BF16 ? 2 : 4) * kHeadDim;
    }
    p.copies = copies;
    p.flag = flag;
    p.H_kv = sh.H_kv;
    p.num_pages = sh.num_pages;
    p.ps = sh.page_size;
    copy_pages_kernel<<<dim3(static_cast<unsigned>(n * sh.H_kv), q4 ? 4 : 2), 256, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
