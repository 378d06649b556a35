// tree_rows.cu -- attention of drafted trees in fp32: every row and key type, on the
// CUDA cores, and the merge of key ranges.
//
// For a (sequence, kv head) with rows r = (query head of the group, draft l)
//   out_r = sum_k softmax(scale * q_r . K_k)[k] V_k
// over the keys before the drafts and the drafts n in the mask of l.
//
// A CTA takes 8 TR rows over a range of the keys, 64 keys at a time; warp w has rows
// TR w .. TR w + TR - 1 to itself: lanes over keys for the scores (2 keys a lane, the row
// values broadcast), lanes over dims for P V (4 dims a lane, the weights broadcast), so
// the softmax needs no barrier.  K of the next keys is on its way during P V, V of these
// during the scores.  Bound by the FMA pipe and shared memory (TR = 8: 16 FMAs for each
// 16-byte load of a key).
#include <algorithm>
#include "tree.h"
#include "ptx.cuh"
#include "q4.cuh"
#include "stage.cuh"

namespace pa {
namespace {

constexpr int kD = kHeadDim;
constexpr int kKeys = 64;           // keys of a step
constexpr int kStride = kD + 4;     // floats of a K row in shared memory: lanes hit all banks
constexpr int kTargetCtas = 4;      // CTAs per SM that key ranges are cut for
constexpr int kMinRange = 256;      // least keys of a range

struct RowsParams {
    const void* q;
    const void *kc, *vc;
    const uint8_t *ks, *vs;
    const int32_t* bt;
    const int32_t* ctx;
    const uint32_t* mask;
    void* out;
    float2* part_ml;  // [(b, kvh, row block)][split][row]
    float* part_o;
    uint32_t* flag;
    int B, H_kv, R, L, W, nrc, nsplit, num_pages, ps, max_npg;
    long long max_S;
    float scale_log2;
};

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ int tree_len(const RowsParams& p, int b, bool& bad) {
    const int S = __ldg(p.ctx + b);
    bad = S < p.L || static_cast<long long>(S) > p.max_S;
    return bad ? 0 : S;
}

// Keys of a range: equal shares in whole steps.
__device__ __forceinline__ int range_keys(int S, int nsplit) {
    return ((S + nsplit - 1) / nsplit + kKeys - 1) / kKeys * kKeys;
}

template <bool F32Q>
__device__ __forceinline__ void store4(void* out, long long at, float4 v) {
    if constexpr (F32Q)
        *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = v;
    else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

enum Rows { kRowsBf16, kRowsF32, kRowsQ4 };

// 64 rows of K or V as fp32 in shared memory; rows of no key are zeros.
template <Rows P>
__device__ __forceinline__ void stage_rows(float* dst, int stride, const void* pool, const uint8_t* scales, const int* rows) {
    const int tid = threadIdx.x;
    if constexpr (P == kRowsF32) {
#pragma unroll
        for (int i = 0; i < kKeys * 32 / 256; ++i) {
            const int r = (tid + 256 * i) >> 5, c = tid & 31, row = rows[r];
            cp_async16(smem_u32(dst + r * stride + 4 * c),
                       static_cast<const float*>(pool) + (row < 0 ? 0 : static_cast<long long>(row) * kD) + 4 * c, row >= 0);
        }
    } else if constexpr (P == kRowsBf16) {
#pragma unroll
        for (int i = 0; i < kKeys * 16 / 256; ++i) {
            const int r = (tid + 256 * i) >> 4, c = tid & 15, row = rows[r];
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (row >= 0) v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(pool) + static_cast<long long>(row) * kD) + c);
            const float2 a = bf16x2_to_float2(v.x), b = bf16x2_to_float2(v.y), d = bf16x2_to_float2(v.z), e = bf16x2_to_float2(v.w);
            float4* const to = reinterpret_cast<float4*>(dst + r * stride + 8 * c);
            to[0] = make_float4(a.x, a.y, b.x, b.y);
            to[1] = make_float4(d.x, d.y, e.x, e.y);
        }
    } else {
        const int r = tid >> 2, c = tid & 3, row = rows[r];  // 32 dims
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        uint32_t s = 0u;
        if (row >= 0) {
            v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(pool) + static_cast<long long>(row) * kQ4CodeBytes) + c);
            s = __ldg(reinterpret_cast<const uint16_t*>(scales + static_cast<long long>(row) * kQ4Groups) + c);
        }
        const float2 sc = f16x2_to_float2(e4m3x2_to_f16x2(s));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t h[4];
            e2m1x8_to_f16x2(w[j], h);
            const float f = j < 2 ? sc.x : sc.y;
            float4* const to = reinterpret_cast<float4*>(dst + r * stride + 32 * c + 8 * j);
            const float2 a = f16x2_to_float2(h[0]), b = f16x2_to_float2(h[1]), d = f16x2_to_float2(h[2]), e = f16x2_to_float2(h[3]);
            to[0] = make_float4(a.x * f, a.y * f, b.x * f, b.y * f);
            to[1] = make_float4(d.x * f, d.y * f, e.x * f, e.y * f);
        }
    }
}

template <int TR>
constexpr int rows_smem() {
    return (8 * TR * kD + kKeys * kStride + kKeys * kD + 8 * TR * kKeys) * 4;
}

template <int TR, bool F32Q, Rows P>
__global__ void __launch_bounds__(256) tree_rows_kernel(const RowsParams p) {
    constexpr int MR = 8 * TR;
    extern __shared__ float smem[];
    float* const qs = smem;                   // [MR][D], scaled
    float* const kb = qs + MR * kD;           // [64][kStride]
    float* const vb = kb + kKeys * kStride;   // [64][D]
    float* const pb = vb + kKeys * kD;        // [MR][64]
    __shared__ int rows[2][kKeys];            // pool rows of a step's keys, -1: none
    __shared__ uint32_t drafted[kTreeMax / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_launch_dependents();

    const long long item = blockIdx.x;
    const int split = static_cast<int>(item % p.nsplit);
    const long long seg = item / p.nsplit;
    const int rc = static_cast<int>(seg % p.nrc);
    const long long bk = seg / p.nrc;
    const int b = static_cast<int>(bk / p.H_kv), kvh = static_cast<int>(bk - static_cast<long long>(b) * p.H_kv);
    bool bad;
    const int S = tree_len(p, b, bad);
    if (bad && tid == 0) atomicOr(p.flag, PA_FLAG_BAD_CONTEXT);
    const int n = range_keys(S, p.nsplit), k0 = min(S, split * n), k1 = min(S, k0 + n), first = S - p.L;

    // which slots hold a draft: nobody sees the others
    if (tid < kTreeMax / 32) drafted[tid] = 0u;
    __syncthreads();
    for (int i = tid; i < p.L && !bad; i += 256) {
        const uint32_t* const m = p.mask + (static_cast<long long>(b) * p.L + i) * p.W;
        uint32_t any = 0u;
        for (int w = 0; w < p.W; ++w) any |= __ldg(m + w);
        if (any) atomicOr(&drafted[i >> 5], 1u << (i & 31));
    }
    // query rows, scaled
    const int r0 = rc * MR;
    const long long qrow = bk * p.R + r0;
    for (int i = tid; i < MR * kD / 4; i += 256) {
        const int r = i / (kD / 4), c = i % (kD / 4);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r0 + r < p.R) {
            if constexpr (F32Q) {
                v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + (qrow + r) * kD) + c);
            } else {
                const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.q) + (qrow + r) * kD) + c);
                const float2 a = bf16x2_to_float2(w.x), e = bf16x2_to_float2(w.y);
                v = make_float4(a.x, a.y, e.x, e.y);
            }
        }
        reinterpret_cast<float4*>(qs)[i] = make_float4(v.x * p.scale_log2, v.y * p.scale_log2, v.z * p.scale_log2, v.w * p.scale_log2);
    }
    __syncthreads();

    auto lookup = [&](int key0, int slot) {  // 64 threads
        const int key = key0 + tid;
        int row = -1;
        if (key < k1) {
            const int i = key - first, lp = key / p.ps;
            const int page = __ldg(p.bt + static_cast<long long>(b) * p.max_npg + lp);
            if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages))
                atomicOr(p.flag, PA_FLAG_BAD_PAGE);
            else if (i < 0 || (drafted[i >> 5] >> (i & 31) & 1u))
                row = (page * p.H_kv + kvh) * p.ps + key - lp * p.ps;
        }
        rows[slot][tid] = row;
    };

    float m[TR], l[TR], o[TR][4];
    bool live[TR];
    int draft[TR];
#pragma unroll
    for (int i = 0; i < TR; ++i) {
        m[i] = neg_inf();
        l[i] = 0.f;
        o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        const int r = r0 + warp * TR + i;
        draft[i] = r % p.L;
        live[i] = r < p.R && !bad && (drafted[draft[i] >> 5] >> (draft[i] & 31) & 1u);
    }
    float* const pw = pb + warp * TR * kKeys;
    const float* const qw = qs + warp * TR * kD;
    if (k0 < k1) {
        if (tid < kKeys) lookup(k0, 0);
        __syncthreads();
        stage_rows<P>(kb, kStride, p.kc, p.ks, rows[0]);
        cp_async_commit();
    }
    for (int key0 = k0, step = 0; key0 < k1; key0 += kKeys, ++step) {
        const int slot = step & 1;
        stage_rows<P>(vb, kD, p.vc, p.vs, rows[slot]);
        cp_async_commit();
        if (key0 + kKeys < k1 && tid < kKeys) lookup(key0 + kKeys, slot ^ 1);
        cp_async_wait<1>();
        __syncthreads();
        // scores of keys lane and lane + 32
        float s[TR][2];
#pragma unroll
        for (int i = 0; i < TR; ++i) s[i][0] = s[i][1] = 0.f;
        const float4* const ka = reinterpret_cast<const float4*>(kb + lane * kStride);
        const float4* const kc = reinterpret_cast<const float4*>(kb + (lane + 32) * kStride);
#pragma unroll 4
        for (int d = 0; d < kD / 4; ++d) {
            const float4 a = ka[d], c = kc[d];
#pragma unroll
            for (int i = 0; i < TR; ++i) {
                const float4 q = *reinterpret_cast<const float4*>(qw + i * kD + 4 * d);
                s[i][0] += q.x * a.x;
                s[i][1] += q.x * c.x;
                s[i][0] += q.y * a.y;
                s[i][1] += q.y * c.y;
                s[i][0] += q.z * a.z;
                s[i][1] += q.z * c.z;
                s[i][0] += q.w * a.w;
                s[i][1] += q.w * c.w;
            }
        }
        const bool tail = key0 + kKeys > first;  // drafts, or past the end
#pragma unroll
        for (int i = 0; i < TR; ++i) {
            if (tail) {
                const uint32_t* const w = p.mask + (static_cast<long long>(b) * p.L + draft[i]) * p.W;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int key = key0 + lane + 32 * h, x = key - first;
                    bool see = key < k1;
                    if (see && x >= 0) see = live[i] && (__ldg(w + (x >> 5)) & drafted[x >> 5]) >> (x & 31) & 1u;
                    if (!see) s[i][h] = neg_inf();
                }
            }
            float mt = fmaxf(s[i][0], s[i][1]);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, d));
            const float mn = fmaxf(m[i], mt), mu = mn == neg_inf() ? 0.f : mn;
            const float alpha = fast_exp2(m[i] - mu), p0 = fast_exp2(s[i][0] - mu), p1 = fast_exp2(s[i][1] - mu);
            m[i] = mn;
            l[i] = l[i] * alpha + (p0 + p1);
#pragma unroll
            for (int d = 0; d < 4; ++d) o[i][d] *= alpha;
            pw[i * kKeys + lane] = p0;
            pw[i * kKeys + lane + 32] = p1;
        }
        cp_async_wait<0>();
        __syncthreads();  // V is there, K is used up
        if (key0 + kKeys < k1) stage_rows<P>(kb, kStride, p.kc, p.ks, rows[slot ^ 1]);
        cp_async_commit();
#pragma unroll 2
        for (int k = 0; k < kKeys; k += 4) {
            float4 v[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) v[x] = *reinterpret_cast<const float4*>(vb + (k + x) * kD + 4 * lane);
#pragma unroll
            for (int i = 0; i < TR; ++i) {
                const float4 w = *reinterpret_cast<const float4*>(pw + i * kKeys + k);
                const float wx[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    o[i][0] += wx[x] * v[x].x;
                    o[i][1] += wx[x] * v[x].y;
                    o[i][2] += wx[x] * v[x].z;
                    o[i][3] += wx[x] * v[x].w;
                }
            }
        }
        __syncthreads();  // V is used up
    }
    cp_async_wait<0>();
#pragma unroll
    for (int i = 0; i < TR; ++i) {
        float sum = l[i];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        const int r = warp * TR + i;
        if (r0 + r >= p.R) continue;
        if (!live[i]) sum = 0.f;
        if (p.nsplit == 1) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;  // (0: a row without keys; NaN stays)
            float4 v = make_float4(o[i][0] * inv, o[i][1] * inv, o[i][2] * inv, o[i][3] * inv);
            if (!live[i]) v = make_float4(0.f, 0.f, 0.f, 0.f);
            store4<F32Q>(p.out, (qrow + r) * kD + 4 * lane, v);
        } else {
            const long long slot = item * MR + r;
            if (lane == 0) p.part_ml[slot] = make_float2(m[i], sum);
            if (sum != 0.f)
                *reinterpret_cast<float4*>(p.part_o + slot * kD + 4 * lane) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
        }
    }
}

// Joins the ranges of a row, a warp per row, four partial states in flight.
template <bool F32Q>
__global__ void __launch_bounds__(256) tree_join_kernel(const RowsParams p, int MR) {
    pdl_wait_primary();
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (row >= static_cast<long long>(p.B) * p.H_kv * p.R) return;
    const long long bk = row / p.R;
    const int r = static_cast<int>(row - bk * p.R), rc = r / MR;
    const long long seg = bk * p.nrc + rc;
    float M = neg_inf(), l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < p.nsplit; k += 4) {
        float2 v[4];
        float4 x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            v[u] = make_float2(neg_inf(), 0.f);
            if (k + u >= p.nsplit) continue;
            const long long slot = (seg * p.nsplit + k + u) * MR + (r - rc * MR);
            v[u] = p.part_ml[slot];
            x[u] = *reinterpret_cast<const float4*>(p.part_o + slot * kD + 4 * lane);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (v[u].y == 0.f) continue;  // no key (x was not written)
            const float mx = fmaxf(M, v[u].x), a = fast_exp2(M - mx), e = fast_exp2(v[u].x - mx);
            M = mx;
            l = l * a + v[u].y * e;
            acc.x = acc.x * a + x[u].x * e;
            acc.y = acc.y * a + x[u].y * e;
            acc.z = acc.z * a + x[u].z * e;
            acc.w = acc.w * a + x[u].w * e;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    store4<F32Q>(p.out, row * kD + 4 * lane, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
}

struct RowsPlan {
    int TR, nrc, nsplit;
    long long segs;
    size_t ml_off, o_off, total;
};

RowsPlan plan(const pa_shape& sh, int sm_count) {
    RowsPlan t;
    const long long R = static_cast<long long>(sh.H_q / sh.H_kv) * sh.L;
    t.TR = R <= 8 ? 1 : R <= 16 ? 2 : R <= 32 ? 4 : 8;
    t.nrc = static_cast<int>((R + 8 * t.TR - 1) / (8 * t.TR));
    t.segs = static_cast<long long>(sh.B) * sh.H_kv * t.nrc;
    const long long cap = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    t.nsplit = static_cast<int>(std::max(1ll, std::min(static_cast<long long>(sm_count) * kTargetCtas / t.segs, cap / kMinRange)));
    // (at most sm_count * kTargetCtas items hold partial states, whatever the shape)
    const size_t slots = static_cast<size_t>(sm_count) * kTargetCtas * 8 * t.TR;
    t.ml_off = kFlagBytes;
    t.o_off = align_up(t.ml_off + slots * 8, 256);
    t.total = t.o_off + slots * kD * 4;
    return t;
}

template <int TR, bool F32Q, Rows P>
pa_status launch_rows(const RowsParams& p, const RowsPlan& t, const TreeCall& c) {
    static int attr_done[64] = {0};
    if (!attr_done[c.dev.device]) {
        if (cudaFuncSetAttribute(tree_rows_kernel<TR, F32Q, P>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 rows_smem<TR>()) != cudaSuccess)
            return PA_ERR_CUDA;
        attr_done[c.dev.device] = 1;
    }
    tree_rows_kernel<TR, F32Q, P><<<static_cast<unsigned>(t.segs * t.nsplit), 256, rows_smem<TR>(), c.stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
    if (t.nsplit == 1) return PA_OK;
    const unsigned grid = static_cast<unsigned>((static_cast<long long>(p.B) * p.H_kv * p.R + 7) / 8);
    return launch_dependent(tree_join_kernel<F32Q>, dim3(grid), 256, 0, c.stream, p, 8 * TR) ? PA_OK : PA_ERR_CUDA;
}

template <bool F32Q, Rows P>
pa_status launch_tr(const RowsParams& p, const RowsPlan& t, const TreeCall& c) {
    switch (t.TR) {
        case 1: return launch_rows<1, F32Q, P>(p, t, c);
        case 2: return launch_rows<2, F32Q, P>(p, t, c);
        case 4: return launch_rows<4, F32Q, P>(p, t, c);
        default: return launch_rows<8, F32Q, P>(p, t, c);
    }
}

}  // namespace

size_t tree_rows_workspace_bytes(const pa_shape& sh, int sm_count) { return plan(sh, sm_count).total; }

pa_status tree_rows_launch(const TreeCall& c) {
    const pa_shape& sh = c.sh;
    const RowsPlan t = plan(sh, c.dev.sm_count);
    uint8_t* const ws = static_cast<uint8_t*>(c.ws);
    RowsParams p;
    p.q = c.q;
    p.kc = c.kc;
    p.vc = c.vc;
    p.ks = static_cast<const uint8_t*>(c.ks);
    p.vs = static_cast<const uint8_t*>(c.vs);
    p.bt = c.bt;
    p.ctx = c.ctx;
    p.mask = c.mask;
    p.out = c.out;
    p.part_ml = reinterpret_cast<float2*>(ws + t.ml_off);
    p.part_o = reinterpret_cast<float*>(ws + t.o_off);
    p.flag = reinterpret_cast<uint32_t*>(ws);
    p.B = sh.B;
    p.H_kv = sh.H_kv;
    p.R = sh.H_q / sh.H_kv * sh.L;
    p.L = sh.L;
    p.W = tree_words(sh.L);
    p.nrc = t.nrc;
    p.nsplit = t.nsplit;
    p.num_pages = sh.num_pages;
    p.ps = sh.page_size;
    p.max_npg = sh.max_pages_per_seq;
    p.max_S = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    p.scale_log2 = c.scale * 1.4426950408889634f;
    if (sh.dtype == PA_F32)
        return c.ks ? launch_tr<true, kRowsQ4>(p, t, c) : launch_tr<true, kRowsF32>(p, t, c);
    return c.ks ? launch_tr<false, kRowsQ4>(p, t, c) : launch_tr<false, kRowsBf16>(p, t, c);
}

}  // namespace pa
