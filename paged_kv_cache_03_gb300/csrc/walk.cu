// walk.cu -- attention over 4-bit pages, and attention that also accumulates
// each key's weight, over 4-bit or bf16 pages.
//
// For a (sequence, kv head) with rows r = (query head of the group, position)
//   s[r][k] = scale * q_r . K_k  (k <= position's frontier),
//   out_r = sum_k softmax(s_r)[k] V_k,   w_out[k] = w_in[k] + sum_r softmax(s_r)[k].
//
// Layout.  A CTA of four warps takes up to 8 * NT rows of one (sequence, kv
// head) over one chunk of its keys; each warp takes every fourth step of 32
// keys (16 over bf16 pages) with its own running max, sum and O, and the warps merge at the end.
// Chunks of one row are merged by walk_combine_kernel.
//
// Keys are the M side of both products: S^T = K Q^T and O^T += V^T P^T with
// mma m16n8k16 (16 keys, 8 rows), so 8 rows fill an instruction and a
// dequantised key serves all of a CTA's rows.  The order of the dims inside a
// contraction is free as long as Q has the same, so lane 4g + t loads 16
// consecutive bytes of key g's code row (dims 32t .. 32t + 31), straight from
// global memory into the A fragments of all 8 k-steps; for V^T it loads the 8
// bytes of dims 16g .. 16g + 15 of keys 2t, 2t + 1, 2t + 8, 2t + 9, which
// share one scale each.  A 4-bit value is exact in f16, so the products see
// exactly the stored values; the query rows are scaled by a power of two into
// f16's range (bf16 keeps all bits; fp32 is split into two f16 parts) and P is
// rounded to f16 (2^-12 relative; split in two for fp32).  Over bf16 pages the
// operands are bf16, and the row sum that divides O adds the rounded weights.
// Max, sums and O are fp32.  The running max moves only when it grows by more
// than 2^8, so O is rarely rescaled.
//
// Weights: walk_weights_kernel repeats K Q^T for 16 keys a warp over all rows
// with the row's final log-sum-exp and adds the rows' probabilities in a fixed
// order (no atomics: a call's results repeat bit for bit).
#include <cfloat>
#include <climits>

#include "cache.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace pa {
namespace {

constexpr int kD = kHeadDim;
constexpr int kWarps = 4;
constexpr float kLazyRescaleLog2 = 8.0f;
constexpr int kMerge = kD + 4;  // floats per (warp, row) in the merge buffer

struct WalkParams {
    const void* q;
    const void *kc, *vc, *ks, *vs;
    const int32_t* bt;
    const int32_t* ctx;
    void* out;
    float4* part_ml;  // [(b, kvh, row)][chunk]: max, sum of the applied weights, sum
    float* part_o;    // [(b, kvh, row)][chunk][D]
    float* lse;       // [(b, kvh, row)] log2 of the sum of 2^score, or null
    const float* w_in;
    float* w_out;
    long long w_S;
    uint32_t* flag;
    int B, H_kv, L, R, num_pages, ps, max_npg, causal, nrc, nkc, C;
    long long max_S;
    float scale_log2;
};

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// The length of sequence b, 0 where it breaks the contract.
__device__ __forceinline__ int seq_len(const WalkParams& p, int b, bool report) {
    const int S = __ldg(p.ctx + b);
    const bool bad = S < 1 || static_cast<long long>(S) > p.max_S || (p.causal && S < p.L);
    if (bad && report) atomicOr(p.flag, PA_FLAG_BAD_CONTEXT);
    return bad ? 0 : S;
}

// Page of logical page lp of sequence b, -1 past `end` (its number of pages)
// and for a bad id (flagged).
__device__ __forceinline__ int page_of(const WalkParams& p, int b, int lp, int end) {
    if (lp >= end) return -1;
    const int pp = __ldg(p.bt + static_cast<long long>(b) * p.max_npg + lp);
    if (pp < 0 || pp >= p.num_pages) {
        atomicOr(p.flag, PA_FLAG_BAD_PAGE);
        return -1;
    }
    return pp;
}

// Pool rows of the 16 U keys of a warp's step (U = 1 or 2); -1: no row (the key
// reads as zeros).  Pages of a multiple of 16 slots: 16 keys share a page, so one row
// number serves them (A16).  Otherwise each lane looks its key up.
template <bool A16, int U>
struct StepRows {
    int r[A16 ? U : 1];
    // row of key i (0 .. 15) of half u
    __device__ __forceinline__ int row(int u, int i) const {
        if constexpr (A16)
            return r[u] + i;
        else
            return __shfl_sync(0xffffffffu, r[0], 16 * u + i);
    }
    __device__ __forceinline__ bool any(int u) const { return A16 ? r[u] >= 0 : true; }
};

// Walks a warp's steps, `stride` keys apart, without dividing.
template <bool A16, int U>
struct StepWalker {
    int lp, slot, dlp, dslot;  // of the step's first key (A16) or this lane's key
    __device__ __forceinline__ void start(const WalkParams& p, int key, int stride) {
        lp = key / p.ps;
        slot = key - lp * p.ps;
        dlp = stride / p.ps;
        dslot = stride - dlp * p.ps;
    }
    __device__ __forceinline__ void next(const WalkParams& p) {
        lp += dlp;
        slot += dslot;
        if (slot >= p.ps) {
            slot -= p.ps;
            ++lp;
        }
    }
    // pages of the step (npg: pages of the sequence)
    __device__ __forceinline__ void pages(const WalkParams& p, int b, int npg, int (&pg)[2]) const {
        pg[0] = page_of(p, b, lp, npg);
        if constexpr (A16 && U == 2) pg[1] = slot + 16 < p.ps ? pg[0] : page_of(p, b, lp + 1, npg);
    }
    __device__ __forceinline__ StepRows<A16, U> rows(const WalkParams& p, int kvh, const int (&pg)[2]) const {
        StepRows<A16, U> w;
        w.r[0] = pg[0] < 0 ? -1 : (pg[0] * p.H_kv + kvh) * p.ps + slot;
        if constexpr (A16 && U == 2) {
            const int s1 = slot + 16 < p.ps ? slot + 16 : 0;
            w.r[1] = pg[1] < 0 ? -1 : (pg[1] * p.H_kv + kvh) * p.ps + s1;
        }
        return w;
    }
};

// ---- 16 keys of 4-bit pages as A fragments --------------------------------
struct Q4Keys {
    static constexpr bool kF16 = true;
    static constexpr int kU = 2;  // 16-key halves per warp step
    // first of the two dims of B fragment register `half` in k-step j, lane t
    __device__ static int qdim(int j, int half, int t) { return 32 * t + 4 * j + 2 * half; }
    uint32_t w[2][4], s[2];
    template <bool A16, int U>
    __device__ __forceinline__ void load(const WalkParams& p, const StepRows<A16, U>& rows, int u, int g, int t) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const long long r = rows.row(u, g + 8 * e);
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            s[e] = 0u;
            if (A16 ? rows.any(u) : r >= 0) {
                x = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.kc) + r * kQ4CodeBytes) + t);
                s[e] = __ldg(reinterpret_cast<const unsigned short*>(static_cast<const uint8_t*>(p.ks) + r * kQ4Groups) + t);
            }
            w[e][0] = x.x;
            w[e][1] = x.y;
            w[e][2] = x.z;
            w[e][3] = x.w;
        }
    }
    // the scales of dims 32t .., 32t + 16 .. of both keys, ready for frags()
    struct Scales {
        uint32_t v[2][2];
    };
    __device__ __forceinline__ Scales scales() const {
        Scales r;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t s2 = e4m3x2_to_f16x2(s[e]);
            r.v[e][0] = __byte_perm(s2, s2, 0x1010);
            r.v[e][1] = __byte_perm(s2, s2, 0x3232);
        }
        return r;
    }
    // A fragments of k-steps 2i and 2i + 1 (code word i of each key)
    __device__ __forceinline__ void frags(const Scales& sc, int i, uint32_t (&a)[2][4]) const {
        uint32_t v0[4], v1[4];
        e2m1x8_to_f16x2(w[0][i], v0);
        e2m1x8_to_f16x2(w[1][i], v1);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            a[j][0] = hmul2(v0[2 * j], sc.v[0][i >> 1]);
            a[j][1] = hmul2(v1[2 * j], sc.v[1][i >> 1]);
            a[j][2] = hmul2(v0[2 * j + 1], sc.v[0][i >> 1]);
            a[j][3] = hmul2(v1[2 * j + 1], sc.v[1][i >> 1]);
        }
    }
};

struct Q4Values {
    uint32_t w[4][2], s[4];
    // keys 2t, 2t + 1, 2t + 8, 2t + 9
    template <bool A16, int U>
    __device__ __forceinline__ void load(const WalkParams& p, const StepRows<A16, U>& rows, int u, int g, int t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const long long r = rows.row(u, 2 * t + (e & 1) + 8 * (e >> 1));
            uint2 x = make_uint2(0u, 0u);
            s[e] = 0u;
            if (A16 ? rows.any(u) : r >= 0) {
                x = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.vc) + r * kQ4CodeBytes) + g);
                s[e] = __ldg(static_cast<const uint8_t*>(p.vs) + r * kQ4Groups + g);
            }
            w[e][0] = x.x;
            w[e][1] = x.y;
        }
    }
    // keys of the half from number n on read as zeros
    __device__ __forceinline__ void cut(int n, int t) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (2 * t + (e & 1) + 8 * (e >> 1) >= n) w[e][0] = w[e][1] = s[e] = 0u;
    }
    struct Scales {
        uint32_t v[2];
    };
    __device__ __forceinline__ Scales scales() const {
        Scales r;
        r.v[0] = e4m3x2_to_f16x2(s[0] | (s[1] << 8));
        r.v[1] = e4m3x2_to_f16x2(s[2] | (s[3] << 8));
        return r;
    }
    // A fragments of m-tiles 4i .. 4i + 3 (code word i of each key); m-tile
    // row g is dim 16g + 2m, row g + 8 dim 16g + 2m + 1
    __device__ __forceinline__ void frags(const Scales& sc, int i, uint32_t (&a)[4][4]) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // keys 2t, 2t + 1; then 2t + 8, 2t + 9
            const uint32_t x = w[2 * h][i], y = w[2 * h + 1][i];
            // bytes (key0 code, key1 code) of the even dims, then of the odd ones
            const uint32_t lo = (x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u);
            const uint32_t hi = ((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u);
            uint32_t vl[4], vh[4];
            e2m1x8_to_f16x2(lo, vl);
            e2m1x8_to_f16x2(hi, vh);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                a[m][2 * h] = hmul2(vl[m], sc.v[h]);
                a[m][2 * h + 1] = hmul2(vh[m], sc.v[h]);
            }
        }
    }
};

// ---- 16 keys of bf16 pages as A fragments ---------------------------------
struct BfKeys {
    static constexpr bool kF16 = false;
    static constexpr int kU = 1;  // (a step of 32 keys would not fit the registers)
    __device__ static int qdim(int j, int half, int t) {
        return 32 * (j >> 1) + 8 * t + 4 * (j & 1) + 2 * half;
    }
    uint4 w[2][4];
    template <bool A16, int U>
    __device__ __forceinline__ void load(const WalkParams& p, const StepRows<A16, U>& rows, int u, int g, int t) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const long long r = rows.row(u, g + 8 * e);
            const bool ok = A16 ? rows.any(u) : r >= 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[e][i] = make_uint4(0u, 0u, 0u, 0u);
                if (ok)
                    w[e][i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.kc) + r * (2 * kD)) + 4 * i + t);
            }
        }
    }
    struct Scales {};
    __device__ __forceinline__ Scales scales() const { return Scales(); }
    __device__ __forceinline__ void frags(const Scales&, int i, uint32_t (&a)[2][4]) const {
        a[0][0] = w[0][i].x;
        a[0][1] = w[1][i].x;
        a[0][2] = w[0][i].y;
        a[0][3] = w[1][i].y;
        a[1][0] = w[0][i].z;
        a[1][1] = w[1][i].z;
        a[1][2] = w[0][i].w;
        a[1][3] = w[1][i].w;
    }
};

struct BfValues {
    uint32_t w[4][8];
    template <bool A16, int U>
    __device__ __forceinline__ void load(const WalkParams& p, const StepRows<A16, U>& rows, int u, int g, int t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const long long r = rows.row(u, 2 * t + (e & 1) + 8 * (e >> 1));
            uint4 x[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
            if (A16 ? rows.any(u) : r >= 0) {
                const uint4* const src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.vc) + r * (2 * kD)) + 2 * g;
                x[0] = __ldg(src);
                x[1] = __ldg(src + 1);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                w[e][4 * i] = x[i].x;
                w[e][4 * i + 1] = x[i].y;
                w[e][4 * i + 2] = x[i].z;
                w[e][4 * i + 3] = x[i].w;
            }
        }
    }
    __device__ __forceinline__ void cut(int n, int t) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (2 * t + (e & 1) + 8 * (e >> 1) >= n) {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[e][i] = 0u;
            }
    }
    struct Scales {};
    __device__ __forceinline__ Scales scales() const { return Scales(); }
    __device__ __forceinline__ void frags(const Scales&, int i, uint32_t (&a)[4][4]) const {
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t x = w[2 * h][4 * i + m], y = w[2 * h + 1][4 * i + m];
                a[m][2 * h] = __byte_perm(x, y, 0x5410);      // dim 2m' of both keys
                a[m][2 * h + 1] = __byte_perm(x, y, 0x7632);  // dim 2m' + 1
            }
    }
};

template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        mma_16816_f16(d, a, b0, b1);
    else
        mma_16816(d, a, b0, b1);
}

// The B fragments of 8 query rows.  Lane 4g + t holds row g; hi and, for fp32
// queries, lo parts.
template <class Keys, bool F32>
struct QueryFrags {
    uint32_t hi[8][2];
    uint32_t lo[F32 ? 8 : 1][2];

    // Loads row `row` of the (b, kvh) block (zeros when !ok); returns the
    // factor that takes a product with the stored fragments to the real one.
    __device__ __forceinline__ float load(const void* q, long long row, bool ok, int t) {
        float2 f[16];
        if constexpr (F32) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                f[k] = make_float2(0.f, 0.f);
                if (ok)
                    f[k] = __ldg(reinterpret_cast<const float2*>(static_cast<const float*>(q) + row * kD +
                                                                 Keys::qdim(k >> 1, k & 1, t)));
            }
        } else {
            uint32_t u[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                u[k] = 0u;
                if (ok)
                    u[k] = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(q) + row * kD +
                                                                   Keys::qdim(k >> 1, k & 1, t)));
            }
            if constexpr (!Keys::kF16) {
#pragma unroll
                for (int k = 0; k < 16; ++k) hi[k >> 1][k & 1] = u[k];
                return 1.f;
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) f[k] = bf16x2_to_float2(u[k]);
        }
        // into f16's range: the row's largest value into [2^14, 2^15)
        float mx = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) mx = fmaxf(mx, fmaxf(fabsf(f[k].x), fabsf(f[k].y)));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int e = static_cast<int>(__float_as_uint(mx) >> 23) - 127;  // -127: zero or subnormal
        const int k2 = e >= 128 ? 0 : min(14 - e, 126);                   // inf or NaN: as they are
        const float up = __uint_as_float(static_cast<uint32_t>(127 + k2) << 23);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - k2) << 23);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float x = f[k].x * up, y = f[k].y * up;
            const uint32_t h = pack_f16x2(x, y);
            hi[k >> 1][k & 1] = h;
            if constexpr (F32) {
                const float2 b = f16x2_to_float2(h);
                lo[k >> 1][k & 1] = pack_f16x2(x - b.x, y - b.y);
            }
        }
        return down;
    }
};

// ---------------------------------------------------------------------------
template <class Keys, class Values, int NT, bool F32, bool A16>
__global__ void __launch_bounds__(kWarps * 32) walk_kernel(const WalkParams p) {
    constexpr bool F16 = Keys::kF16;
    constexpr int ROWS = 8 * NT;
    constexpr int U = Keys::kU, kStep = 16 * U;
    extern __shared__ float merge[];  // [warp][row][kMerge]: o, m, applied sum, sum
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    int item = static_cast<int>(blockIdx.x);
    const int kc = item % p.nkc;
    item /= p.nkc;
    const int rc = item % p.nrc;
    item /= p.nrc;
    const int kvh = item % p.H_kv, b = item / p.H_kv;
    const int S = seq_len(p, b, kc == 0 && rc == 0 && kvh == 0 && threadIdx.x == 0);
    const int r0 = rc * ROWS, nrows = min(ROWS, p.R - r0);
    const long long row0 = (static_cast<long long>(b) * p.H_kv + kvh) * p.R + r0;

    // the last key each of this lane's rows (2t, 2t + 1 of every n-tile) sees
    int lim[NT][2], lim_min = INT_MAX, lim_max = -1;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int rr = 8 * n + 2 * t + e;
            lim[n][e] = -1;
            if (rr < nrows) lim[n][e] = p.causal ? (r0 + rr) % p.L + S - p.L : S - 1;
            if (rr < nrows) {
                lim_min = min(lim_min, lim[n][e]);
                lim_max = max(lim_max, lim[n][e]);
            }
        }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, o));
        lim_max = max(lim_max, __shfl_xor_sync(0xffffffffu, lim_max, o));
    }
    const int k0 = kc * p.C;
    const int k1 = S > 0 ? min(lim_max + 1, k0 + p.C) : 0;

    QueryFrags<Keys, F32> q[NT];
    float qs[NT][2];  // score scale of rows 2t, 2t + 1 in log2 units
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int rr = 8 * n + g;
        const float down = q[n].load(p.q, row0 + rr, rr < nrows, t);
        // lane 4g' + t' holds row g': rows 2t and 2t + 1 are lanes 8t and 8t + 4
        // (never 0: a hidden key's -inf times it has to stay -inf)
        qs[n][0] = fmaxf(__shfl_sync(0xffffffffu, down, 8 * t) * p.scale_log2, FLT_MIN);
        qs[n][1] = fmaxf(__shfl_sync(0xffffffffu, down, 8 * t + 4) * p.scale_log2, FLT_MIN);
    }

    float m[NT][2], l[NT][2], la[NT][2];
    float o[NT][8][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = neg_inf();
        l[n][0] = l[n][1] = la[n][0] = la[n][1] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
    }

    // The values of a step are requested when it begins and the keys of the next
    // one with them, so a step's S = K Q^T hides both.
    const int npg = (S + p.ps - 1) / p.ps;
    StepWalker<A16, U> wk;
    const int first = k0 + warp * kStep;
    wk.start(p, A16 ? first : first + lane, kWarps * kStep);
    StepRows<A16, U> rows = {};
    int pg[2] = {-1, -1};
    Keys kk[U];
    if (first < k1) {
        wk.pages(p, b, npg, pg);
        rows = wk.rows(p, kvh, pg);
#pragma unroll
        for (int u = 0; u < U; ++u) kk[u].load(p, rows, u, g, t);
        wk.next(p);
        if (first + kWarps * kStep < k1) wk.pages(p, b, npg, pg);
    }
    for (int base = first; base < k1; base += kWarps * kStep) {
        Values vv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) vv[u].load(p, rows, u, g, t);
        Keys kn[U];
        if (base + kWarps * kStep < k1) {
            rows = wk.rows(p, kvh, pg);
#pragma unroll
            for (int u = 0; u < U; ++u) kn[u].load(p, rows, u, g, t);
            wk.next(p);
            if (base + 2 * kWarps * kStep < k1) wk.pages(p, b, npg, pg);
        }
        // S^T: 16 U keys x 8 NT rows
        float s[NT][U][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int u = 0; u < U; ++u) s[n][u][0] = s[n][u][1] = s[n][u][2] = s[n][u][3] = 0.f;
        typename Keys::Scales ksc[U];
#pragma unroll
        for (int u = 0; u < U; ++u) ksc[u] = kk[u].scales();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                uint32_t a[2][4];
                kk[u].frags(ksc[u], i, a);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma<F16>(s[n][u], a[j], q[n].hi[2 * i + j][0], q[n].hi[2 * i + j][1]);
                        if constexpr (F32) mma<F16>(s[n][u], a[j], q[n].lo[2 * i + j][0], q[n].lo[2 * i + j][1]);
                    }
            }
        if (base + kStep - 1 > lim_min) {  // a row does not see every key (uniform over the warp)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (base + 16 * u + g + 8 * (e >> 1) > lim[n][e & 1]) s[n][u][e] = neg_inf();
        }
        uint32_t pb[NT][U][2], pl[NT][U][2];  // P^T fragments, and their low parts
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float mt[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
                mt[e] = fmaxf(fmaxf(s[n][0][e], s[n][0][2 + e]), fmaxf(s[n][U - 1][e], s[n][U - 1][2 + e])) * qs[n][e];
            if (__any_sync(0xffffffffu, mt[0] > m[n][0] + kLazyRescaleLog2 || mt[1] > m[n][1] + kLazyRescaleLog2)) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    mt[0] = fmaxf(mt[0], __shfl_xor_sync(0xffffffffu, mt[0], d));
                    mt[1] = fmaxf(mt[1], __shfl_xor_sync(0xffffffffu, mt[1], d));
                }
                const bool g0 = mt[0] > m[n][0] + kLazyRescaleLog2, g1 = mt[1] > m[n][1] + kLazyRescaleLog2;
                const float a0 = g0 ? fast_exp2(m[n][0] - mt[0]) : 1.f;  // 2^-inf = 0 at the start
                const float a1 = g1 ? fast_exp2(m[n][1] - mt[1]) : 1.f;
                if (g0) m[n][0] = mt[0];
                if (g1) m[n][1] = mt[1];
                l[n][0] *= a0;
                l[n][1] *= a1;
                la[n][0] *= a0;
                la[n][1] *= a1;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    o[n][i][0] *= a0;
                    o[n][i][1] *= a1;
                    o[n][i][2] *= a0;
                    o[n][i][3] *= a1;
                }
            }
            const float mu[2] = {m[n][0] == neg_inf() ? 0.f : m[n][0], m[n][1] == neg_inf() ? 0.f : m[n][1]};
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) {  // keys g, then g + 8
                    const float p0 = fast_exp2(fmaf(s[n][u][2 * h], qs[n][0], -mu[0]));
                    const float p1 = fast_exp2(fmaf(s[n][u][2 * h + 1], qs[n][1], -mu[1]));
                    l[n][0] += p0;
                    l[n][1] += p1;
                    if constexpr (F16) {
                        const uint32_t x = pack_f16x2(p0, p1);
                        pb[n][u][h] = movmatrix_trans(x);
                        if constexpr (F32) {
                            const float2 f = f16x2_to_float2(x);
                            pl[n][u][h] = movmatrix_trans(pack_f16x2(p0 - f.x, p1 - f.y));
                        }
                    } else {
                        const uint32_t x = pack_bf16x2(p0, p1);
                        const float2 f = bf16x2_to_float2(x);
                        la[n][0] += f.x;
                        la[n][1] += f.y;
                        pb[n][u][h] = movmatrix_trans(x);
                    }
                }
        }
        if (base + kStep > S) {  // slots past the context may hold anything
#pragma unroll
            for (int u = 0; u < U; ++u) vv[u].cut(S - base - 16 * u, t);
        }
        // O^T += V^T P^T
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const typename Values::Scales vsc = vv[u].scales();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t a[4][4];
                vv[u].frags(vsc, i, a);
#pragma unroll
                for (int mm = 0; mm < 4; ++mm)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma<F16>(o[n][4 * i + mm], a[mm], pb[n][u][0], pb[n][u][1]);
                        if constexpr (F32) mma<F16>(o[n][4 * i + mm], a[mm], pl[n][u][0], pl[n][u][1]);
                    }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) kk[u] = kn[u];
    }

    // ---- merge the four warps ---------------------------------------------
    float* const mw = merge + warp * ROWS * kMerge;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float lt = l[n][e], at = F16 ? l[n][e] : la[n][e];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
                lt += __shfl_xor_sync(0xffffffffu, lt, d);
                at += __shfl_xor_sync(0xffffffffu, at, d);
            }
            float* const mr = mw + (8 * n + 2 * t + e) * kMerge;
            if (g == 0) {
                mr[kD] = m[n][e];
                mr[kD + 1] = at;
                mr[kD + 2] = lt;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)  // dims 16g .. 16g + 15 of the row
                *reinterpret_cast<float4*>(mr + 16 * g + 4 * i) =
                    make_float4(o[n][2 * i][e], o[n][2 * i][2 + e], o[n][2 * i + 1][e], o[n][2 * i + 1][2 + e]);
        }
    __syncthreads();
    const int d = threadIdx.x;  // one dim per thread
    for (int rr = 0; rr < nrows; ++rr) {
        float M = neg_inf();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, merge[(w * ROWS + rr) * kMerge + kD]);
        float acc = 0.f, at = 0.f, lt = 0.f;
        if (M != neg_inf()) {
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float* const mr = merge + (w * ROWS + rr) * kMerge;
                const float a = fast_exp2(mr[kD] - M);
                acc += a * mr[d];
                at += a * mr[kD + 1];
                lt += a * mr[kD + 2];
            }
        }
        const long long row = row0 + rr;
        if (p.nkc == 1) {
            const float v = at > 0.f ? acc / at : 0.f;
            if constexpr (F32)
                static_cast<float*>(p.out)[row * kD + d] = v;
            else
                static_cast<uint16_t*>(p.out)[row * kD + d] = float_to_bf16_bits(v);
            if (d == 0 && p.lse) p.lse[row] = lt > 0.f ? M + log2f(lt) : __int_as_float(0x7f800000);
        } else {
            if (d == 0) p.part_ml[row * p.nkc + kc] = make_float4(M, at, lt, 0.f);
            if (M != neg_inf()) p.part_o[(row * p.nkc + kc) * kD + d] = acc;
        }
    }
}

// Merges the key chunks of a row: one warp per row, four dims per lane.  A
// row without keys is written as zeros.
template <bool F32>
__global__ void __launch_bounds__(128) walk_combine_kernel(const WalkParams p) {
    pdl_wait_primary();
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= static_cast<long long>(p.B) * p.H_kv * p.R) return;
    const int lane = threadIdx.x & 31;
    const float4* const ml = p.part_ml + row * p.nkc;
    const float* const po = p.part_o + row * p.nkc * kD + 4 * lane;
    float M = neg_inf();
    for (int c = lane; c < p.nkc; c += 32) M = fmaxf(M, ml[c].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float at = 0.f, lt = 0.f;
    if (M != neg_inf()) {
        for (int c = 0; c < p.nkc; ++c) {
            const float4 v = ml[c];
            if (v.x == neg_inf()) continue;  // no key: no o row either
            const float a = fast_exp2(v.x - M);
            at += a * v.y;
            lt += a * v.z;
            const float4 x = *reinterpret_cast<const float4*>(po + static_cast<long long>(c) * kD);
            acc.x += a * x.x;
            acc.y += a * x.y;
            acc.z += a * x.z;
            acc.w += a * x.w;
        }
    }
    const float inv = at > 0.f ? 1.f / at : 0.f;
    if constexpr (F32)
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * kD + 4 * lane) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * kD + 4 * lane) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lane == 0 && p.lse) p.lse[row] = lt > 0.f ? M + log2f(lt) : __int_as_float(0x7f800000);
}

// w_out[b, kvh, k] = w_in[b, kvh, k] + the rows' probabilities of key k, 0 past
// the context.  A warp holds 16 keys as A fragments and runs over the rows.
template <class Keys, bool F32>
__global__ void __launch_bounds__(kWarps * 32) walk_weights_kernel(const WalkParams p, int ntile) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    int item = static_cast<int>(blockIdx.x);
    const int tile = item % ntile;
    item /= ntile;
    const int kvh = item % p.H_kv, b = item / p.H_kv;
    const long long base = (static_cast<long long>(tile) * kWarps + warp) * 16;
    const int S = seq_len(p, b, false);
    float acc[2] = {0.f, 0.f};  // keys g and g + 8, this lane's rows
    if (base < S) {
        const int k0 = static_cast<int>(base);
        StepWalker<false, 1> wk;
        wk.start(p, k0 + lane, 0);
        int pg[2];
        wk.pages(p, b, k0 + lane < S && lane < 16 ? INT_MAX : 0, pg);
        const StepRows<false, 1> rows = wk.rows(p, kvh, pg);
        Keys kk;
        kk.load(p, rows, 0, g, t);
        const typename Keys::Scales ksc = kk.scales();
        const long long row0 = (static_cast<long long>(b) * p.H_kv + kvh) * p.R;
        for (int r0 = 0; r0 < p.R; r0 += 8) {
            QueryFrags<Keys, F32> q;
            const float down = q.load(p.q, row0 + r0 + g, r0 + g < p.R, t);
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t a[2][4];
                kk.frags(ksc, i, a);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    mma<Keys::kF16>(s, a[j], q.hi[2 * i + j][0], q.hi[2 * i + j][1]);
                    if constexpr (F32) mma<Keys::kF16>(s, a[j], q.lo[2 * i + j][0], q.lo[2 * i + j][1]);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float qs = fmaxf(__shfl_sync(0xffffffffu, down, 8 * t + 4 * e) * p.scale_log2, FLT_MIN);
                const int r = r0 + 2 * t + e;
                if (r >= p.R) continue;
                const int lim = p.causal ? r % p.L + S - p.L : S - 1;
                const float lse = p.lse[row0 + r];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = g + 8 * h;
                    if (k0 + k <= lim) acc[h] += fast_exp2(s[2 * h + e] * qs - lse);
                }
            }
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        acc[h] += __shfl_xor_sync(0xffffffffu, acc[h], 1);
        acc[h] += __shfl_xor_sync(0xffffffffu, acc[h], 2);
    }
    if (t < 2) {
        const long long k = base + g + 8 * t;
        if (k < p.w_S) {
            const long long at = (static_cast<long long>(b) * p.H_kv + kvh) * p.w_S + k;
            const float old = p.w_in && k < S ? p.w_in[at] : 0.f;
            p.w_out[at] = k < S ? old + (t ? acc[1] : acc[0]) : 0.f;
        }
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
struct WalkPlan {
    int R, nt, nrc, nkc, C;
    size_t ml_off, o_off, lse_off, total;
};

// Rows per CTA: 8, or 16 where a (sequence, kv head) has more than 8 (not for
// fp32 queries, whose fragments take twice the registers).  Key chunks: enough
// for about eight CTAs per SM, of at least 256 keys.
WalkPlan plan(const pa_shape& sh, bool weights, int sm_count) {
    WalkPlan w;
    w.R = sh.H_q / sh.H_kv * sh.L;
    w.nt = w.R > 8 && sh.dtype == PA_BF16 ? 2 : 1;
    w.nrc = (w.R + 8 * w.nt - 1) / (8 * w.nt);
    const long long cap = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    const long long items = static_cast<long long>(sh.B) * sh.H_kv * w.nrc;
    long long nkc = (8ll * sm_count + items - 1) / items;
    const long long most = (cap + 255) / 256;
    nkc = nkc < most ? nkc : most;
    long long C = (cap + nkc - 1) / nkc;
    C = (C + kWarps * 32 - 1) / (kWarps * 32) * (kWarps * 32);  // whole steps of every warp
    w.C = static_cast<int>(C);
    w.nkc = static_cast<int>((cap + C - 1) / C);
    const size_t rows = static_cast<size_t>(sh.B) * sh.H_kv * w.R;
    size_t off = kFlagBytes;
    w.ml_off = off;
    if (w.nkc > 1) off = align_up(off + rows * w.nkc * 16, 256);
    w.o_off = off;
    if (w.nkc > 1) off = align_up(off + rows * w.nkc * kD * 4, 256);
    w.lse_off = off;
    if (weights) off = align_up(off + rows * 4, 256);
    w.total = off;
    return w;
}

template <class Keys, class Values, int NT, bool F32, bool A16>
pa_status launch_as(const WalkParams& p, cudaStream_t stream) {
    constexpr size_t smem = sizeof(float) * kWarps * 8 * NT * kMerge;
    static_assert(smem <= 48 * 1024, "merge buffer within the default limit");
    const long long items = static_cast<long long>(p.B) * p.H_kv * p.nrc * p.nkc;
    const long long rows = static_cast<long long>(p.B) * p.H_kv * p.R;
    const long long ntile = (p.w_S + 16 * kWarps - 1) / (16 * kWarps);
    if (items > INT_MAX || rows > 4ll * INT_MAX || ntile * p.B * p.H_kv > INT_MAX) return PA_ERR_UNSUPPORTED;
    walk_kernel<Keys, Values, NT, F32, A16><<<static_cast<unsigned>(items), kWarps * 32, smem, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
    if (p.nkc > 1) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>((rows + 3) / 4));
        cfg.blockDim = dim3(128);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, walk_combine_kernel<F32>, p) != cudaSuccess) return PA_ERR_CUDA;
    }
    if (p.w_out) {
        walk_weights_kernel<Keys, F32><<<static_cast<unsigned>(ntile * p.B * p.H_kv), kWarps * 32, 0, stream>>>(
            p, static_cast<int>(ntile));
        if (cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
    }
    return PA_OK;
}

template <class Keys, class Values, int NT, bool F32>
pa_status launch(const WalkParams& p, cudaStream_t stream) {
    return p.ps % 16 == 0 ? launch_as<Keys, Values, NT, F32, true>(p, stream)
                          : launch_as<Keys, Values, NT, F32, false>(p, stream);
}

// ---- many rows over 4-bit pages: dense bf16 copies and the tensor-core tiles --
// (exact: a 4-bit value is a bf16 number).  Sequences go in groups whose
// copies fit kDenseBytes.
// Rows per kv head from which the tiles take a call.  Measured (walk, tiles, us;
// G = 4, H_kv = 8): B = 8 over 1000 .. 8000 keys 61, 96 at 32 rows, 91, 96 at 64,
// 123, 97 at 96; B = 1 over 16000 keys 41, 41 at 16, 57, 41 at 32; B = 64 over 500
// .. 2000 keys 111, 166 at 32, 169, 166 at 64.
constexpr int kTileRows = 48;
constexpr size_t kDenseBytes = size_t(1) << 30;

struct TilePlan {
    pa_shape sh;  // one group, over the dense copies
    size_t id_off, k_off, v_off, total;  // id: block table, then lengths
};

bool tiles_take(const pa_shape& sh, bool q4, bool weights, int sm_count, TilePlan* t) {
    if (!q4 || weights || sh.dtype != PA_BF16) return false;
    if (static_cast<long long>(sh.H_q / sh.H_kv) * sh.L < kTileRows) return false;
    const long long cap = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    const long long slots = (cap + 127) / 128 * 128;
    const size_t per_seq = static_cast<size_t>(slots) * sh.H_kv * kD * 2 * 2;
    if (slots * sh.H_kv >= (1ll << 31)) return false;
    long long nb = static_cast<long long>(kDenseBytes / per_seq);
    nb = nb < 1 ? 1 : nb < sh.B ? nb : sh.B;
    t->sh = sh;
    t->sh.B = static_cast<int>(nb);
    t->sh.num_pages = t->sh.B;
    t->sh.page_size = static_cast<int>(slots);
    t->sh.max_pages_per_seq = 1;
    if (!prefill_supported(t->sh)) return false;
    size_t off = tile_partials_offset(t->sh, sm_count) + tile_partial_bytes(t->sh, sm_count);
    pa_shape last = t->sh;  // the last group may split its keys more
    last.B = sh.B % last.B > 0 ? sh.B % last.B : last.B;
    const size_t off_last = tile_partials_offset(last, sm_count) + tile_partial_bytes(last, sm_count);
    t->id_off = off = align_up(off > off_last ? off : off_last, 256);
    off = align_up(off + 8 * static_cast<size_t>(nb), 256);
    t->k_off = off;
    off += nb * per_seq / 2;
    t->v_off = off;
    t->total = off + nb * per_seq / 2;
    return true;
}

pa_status tiles_launch(const WalkCall& c, const TilePlan& t) {
    const pa_shape& sh = c.sh;
    uint8_t* const ws = static_cast<uint8_t*>(c.ws);
    const pa_q4_pool pool = {const_cast<void*>(c.kc), const_cast<void*>(c.ks), const_cast<void*>(c.vc),
                             const_cast<void*>(c.vs)};
    const size_t per_seq = static_cast<size_t>(sh.H_q) * sh.L * kD * 2;  // query and output bytes
    for (int b0 = 0; b0 < sh.B; b0 += t.sh.B) {
        const int nb = t.sh.B < sh.B - b0 ? t.sh.B : sh.B - b0;
        pa_shape src = sh;
        src.B = nb;
        pa_status st = q4_gather_launch(src, pool, c.bt + static_cast<long long>(b0) * sh.max_pages_per_seq,
                                        c.ctx + b0, t.sh.page_size, 0, 0,
                                        reinterpret_cast<int32_t*>(ws + t.id_off), t.sh.B, ws + t.k_off, ws + t.v_off,
                                        reinterpret_cast<uint32_t*>(ws), c.stream);
        if (st != PA_OK) return st;
        Call d;
        d.sh = t.sh;
        d.sh.B = nb;
        d.q = static_cast<const uint8_t*>(c.q) + b0 * per_seq;
        d.kp = ws + t.k_off;
        d.vp = ws + t.v_off;
        d.bt = reinterpret_cast<const int32_t*>(ws + t.id_off);
        d.ctx = d.bt + t.sh.B;
        d.scale = c.scale;
        d.causal = c.causal;
        d.out = static_cast<uint8_t*>(c.out) + b0 * per_seq;
        d.ws = c.ws;
        d.ws_bytes = t.id_off;
        d.stream = c.stream;
        d.dev = c.dev;
        st = prefill_launch(d);
        if (st != PA_OK) return st;
    }
    return PA_OK;
}

}  // namespace

size_t walk_workspace_bytes(const pa_shape& sh, bool q4, bool weights, int sm_count) {
    TilePlan t;
    if (tiles_take(sh, q4, weights, sm_count, &t)) return t.total;
    return plan(sh, weights, sm_count).total;
}

pa_status walk_launch(const WalkCall& c) {
    const pa_shape& sh = c.sh;
    TilePlan t;
    if (tiles_take(sh, c.ks != nullptr, c.w_out != nullptr, c.dev.sm_count, &t)) {
        if (c.ws_bytes < t.total) return PA_ERR_WORKSPACE;
        return tiles_launch(c, t);
    }
    const WalkPlan w = plan(sh, c.w_out != nullptr, c.dev.sm_count);
    if (c.ws_bytes < w.total) return PA_ERR_WORKSPACE;
    uint8_t* const ws = static_cast<uint8_t*>(c.ws);
    WalkParams p;
    p.q = c.q;
    p.kc = c.kc;
    p.vc = c.vc;
    p.ks = c.ks;
    p.vs = c.vs;
    p.bt = c.bt;
    p.ctx = c.ctx;
    p.out = c.out;
    p.part_ml = reinterpret_cast<float4*>(ws + w.ml_off);
    p.part_o = reinterpret_cast<float*>(ws + w.o_off);
    p.lse = c.w_out ? reinterpret_cast<float*>(ws + w.lse_off) : nullptr;
    p.w_in = c.w_in;
    p.w_out = c.w_out;
    p.w_S = c.w_S;
    p.flag = reinterpret_cast<uint32_t*>(ws);
    p.B = sh.B;
    p.H_kv = sh.H_kv;
    p.L = sh.L;
    p.R = w.R;
    p.num_pages = sh.num_pages;
    p.ps = sh.page_size;
    p.max_npg = sh.max_pages_per_seq;
    p.causal = c.causal;
    p.nrc = w.nrc;
    p.nkc = w.nkc;
    p.C = w.C;
    p.max_S = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    p.scale_log2 = c.scale * 1.4426950408889634f;
    if (!c.ks) {
        if (w.nt == 2) return launch<BfKeys, BfValues, 2, false>(p, c.stream);
        return launch<BfKeys, BfValues, 1, false>(p, c.stream);
    }
    if (sh.dtype == PA_F32) return launch<Q4Keys, Q4Values, 1, true>(p, c.stream);
    if (w.nt == 2) return launch<Q4Keys, Q4Values, 2, false>(p, c.stream);
    return launch<Q4Keys, Q4Values, 1, false>(p, c.stream);
}

}  // namespace pa
