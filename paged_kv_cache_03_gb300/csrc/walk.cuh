// walk.cuh -- what the kernels of the cache attention share: the call's
// parameters, page lookups, K/V fragments, equal shares of the keys.
#pragma once
#include <cfloat>
#include <climits>

#include "cache.h"
#include "ptx.cuh"
#include "stage.cuh"

namespace pa {
namespace walk {

constexpr int kD = kHeadDim;
constexpr int kWarps = 4;
constexpr float kLazyRescaleLog2 = 8.0f;
// fp32 queries: a weight is hi + kLowStep * lo, both f16, and V^T lo is scaled before V^T hi
// is added to it.  lo has f16's whole range for itself, steps of 2^-35 where the row's
// largest weight is at least 1: with both parts in one range, keys below 2^-25 of the
// largest counted in the row's sum and were missing in O (32768 of them 2^-25.5 each:
// 3.5e-4 of the result).
constexpr float kLowScale = 2048.f, kLowStep = 1.f / kLowScale;
constexpr int kMerge = kD + 4;  // floats per (warp, row) in the merge buffer

struct WalkParams {
    const void* q;
    const void *kc, *vc, *ks, *vs;
    const int32_t* bt;
    const int32_t* ctx;
    void* out;
    float4* part_ml;  // [2 slots per CTA][ROWS]: max, sum of the applied weights, sum
    float* part_o;    // [2 slots per CTA][ROWS][D]
    int4* split;      // per CTA: the segment that starts in its share and ends in a later one
    float* lse;       // [(b, kvh, row)] log2 of the sum of 2^score, or null
    float* score;     // [(b, kvh)][key < cap][row] scores in log2 units, or null
    long long cap;    // keys of a (b, kvh) in score
    const float* w_in;
    float* w_out;
    long long w_S;
    uint32_t* flag;
    int B, H_kv, L, R, num_pages, ps, max_npg, causal, nrc;
    int whole;    // walk_kernel: 1 one CTA per segment, 0 equal shares of all keys
    int min_per;  // least cost of a share
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

// A page id, requested before it is needed: kNoPage past a sequence's pages.
constexpr int kNoPage = INT_MIN;

// Pool row of slot `slot` of page `pg`, -1 for no page or a bad id; bad ids are
// gathered in `bad` (no branch here) and flagged once at a kernel's end.
__device__ __forceinline__ int row_in(const WalkParams& p, int kvh, int pg, int slot, bool& bad) {
    const bool ok = static_cast<unsigned>(pg) < static_cast<unsigned>(p.num_pages);
    bad |= !ok && pg != kNoPage;
    return ok ? (pg * p.H_kv + kvh) * p.ps + slot : -1;
}
__device__ __forceinline__ void report_pages(const WalkParams& p, bool bad) {
    if (__any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0) atomicOr(p.flag, PA_FLAG_BAD_PAGE);
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
    bool bad = false;          // a bad page id was met
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
    // Requests the step's page ids (npg: pages of the sequence, 0 for a step that
    // is not taken); rows() checks them a step later, so that nothing waits for the
    // load here.
    __device__ __forceinline__ void pages(const int32_t* row, const WalkParams& p, int npg, int (&pg)[2]) const {
        pg[0] = lp < npg ? __ldg(row + lp) : kNoPage;
        if constexpr (A16 && U == 2) pg[1] = slot + 16 >= p.ps && lp + 1 < npg ? __ldg(row + lp + 1) : kNoPage;
    }
    __device__ __forceinline__ StepRows<A16, U> rows(const WalkParams& p, int kvh, const int (&pg)[2]) {
        StepRows<A16, U> w;
        w.r[0] = row_in(p, kvh, pg[0], slot, bad);
        if constexpr (A16 && U == 2)
            w.r[1] = slot + 16 < p.ps ? (w.r[0] < 0 ? -1 : w.r[0] + 16) : row_in(p, kvh, pg[1], 0, bad);
        return w;
    }
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

// ---- a warp's step of keys and values in shared memory ----------------------
// Filled by asynchronous copies, whole lines a warp; the values' rows are placed
// so that the fragment loads below meet no bank conflict.
template <bool Q4>
struct Stage;

template <>
struct Stage<true> {  // 32 keys: K codes, V codes, K scales, V scales
    static constexpr int kV = 2048, kKS = 4096, kVS = 4352, kBytes = 4608;
    // byte of 16-byte chunk c of value i (0 .. 15) of half u
    __device__ static uint32_t v_at(int u, int i, int c) {
        const int slot = (i >> 1) | ((i & 1) << 3);
        return kV + (16 * u + slot) * 64 + ((c ^ (slot & 2)) << 4);
    }
    template <bool A16>
    __device__ static void fill(const WalkParams& p, const StepRows<A16, 2>& rows, uint32_t st, int lane) {
        const uint8_t* const kc = static_cast<const uint8_t*>(p.kc);
        const uint8_t* const vc = static_cast<const uint8_t*>(p.vc);
        const uint8_t* const ks = static_cast<const uint8_t*>(p.ks);
        const uint8_t* const vs = static_cast<const uint8_t*>(p.vs);
        if constexpr (A16) {  // 16 rows lie together: 64 chunks, two copies a lane
            // v_at(u, i, c) of chunk lane + 32 j is v0 + 1024 u + 256 j
            const uint32_t v0 = st + v_at(0, lane >> 2, lane & 3);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const bool ok = rows.any(u);
                const long long off = ok ? static_cast<long long>(rows.r[u]) * kQ4CodeBytes + 16 * lane : 0;
                const uint8_t* const k = kc + off;
                const uint8_t* const v = vc + off;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    cp_async16(st + 16 * lane + 1024 * u + 512 * j, k + 512 * j, ok);
                    cp_async16(v0 + 1024 * u + 256 * j, v + 512 * j, ok);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int u = j >> 1, i = (lane >> 2) + 8 * (j & 1), c = lane & 3;
                const int row = rows.row(u, i);
                const bool ok = row >= 0;
                const long long off = ok ? static_cast<long long>(row) * kQ4CodeBytes + 16 * c : 0;
                cp_async16(st + 16 * (lane + 32 * j), kc + off, ok);
                cp_async16(st + v_at(u, i, c), vc + off, ok);
            }
        }
        if constexpr (A16) {  // two keys a chunk: lanes 0 - 15 K, 16 - 31 V
            const int i = lane & 15, r = i < 8 ? rows.r[0] : rows.r[1];
            const long long off = r >= 0 ? static_cast<long long>(r + 2 * (i & 7)) * kQ4Groups : 0;
            cp_async16(st + kKS + 16 * lane, (lane < 16 ? ks : vs) + off, r >= 0);
        } else {
            const int r = rows.r[0];
            const long long off = r >= 0 ? static_cast<long long>(r) * kQ4Groups : 0;
            cp_async8(st + kKS + 8 * lane, ks + off, r >= 0);
            cp_async8(st + kVS + 8 * lane, vs + off, r >= 0);
        }
    }
};

template <>
struct Stage<false> {  // 16 keys: K rows, V rows
    static constexpr int kV = 4096, kBytes = 8192;
    __device__ static uint32_t k_at(int i, int c) { return i * 256 + ((c ^ ((i & 1) << 2)) << 4); }
    __device__ static uint32_t v_at(int i, int c) {
        return kV + i * 256 + ((c ^ (((i >> 1) & 1) | ((i >> 2 & 1) << 2))) << 4);
    }
    template <bool A16>
    __device__ static void fill(const WalkParams& p, const StepRows<A16, 1>& rows, uint32_t st, int lane) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = (lane >> 4) + 2 * j, c = lane & 15;
            const int row = rows.row(0, i);
            const bool ok = A16 ? rows.any(0) : row >= 0;
            const long long off = ok ? static_cast<long long>(row) * (2 * kD) + 16 * c : 0;
            cp_async16(st + k_at(i, c), static_cast<const uint8_t*>(p.kc) + off, ok);
            cp_async16(st + v_at(i, c), static_cast<const uint8_t*>(p.vc) + off, ok);
        }
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
    __device__ __forceinline__ void load(uint32_t st, int u, int g, int t) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint4 x = lds128(st + (16 * u + g + 8 * e) * 64 + t * 16);
            w[e][0] = x.x;
            w[e][1] = x.y;
            w[e][2] = x.z;
            w[e][3] = x.w;
            s[e] = lds16(st + Stage<true>::kKS + (16 * u + g + 8 * e) * 8 + 2 * t);
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
    __device__ __forceinline__ void load(uint32_t st, int u, int g, int t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 2 * t + (e & 1) + 8 * (e >> 1);
            const uint2 x = lds64(st + Stage<true>::v_at(u, i, g >> 1) + 8 * (g & 1));
            w[e][0] = x.x;
            w[e][1] = x.y;
            s[e] = lds8(st + Stage<true>::kVS + (16 * u + i) * 8 + g);
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
    __device__ __forceinline__ void load(uint32_t st, int, int g, int t) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) w[e][i] = lds128(st + Stage<false>::k_at(g + 8 * e, 4 * i + t));
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
    __device__ __forceinline__ void load(uint32_t st, int, int g, int t) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 x = lds128(st + Stage<false>::v_at(2 * t + (e & 1) + 8 * (e >> 1), 2 * g + i));
                w[e][4 * i] = x.x;
                w[e][4 * i + 1] = x.y;
                w[e][4 * i + 2] = x.z;
                w[e][4 * i + 3] = x.w;
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

// The B fragments of 8 query rows.  Lane 4g + t holds row g; hi and, for fp32
// queries, lo parts.
template <class Keys, bool F32>
struct QueryFrags {
    uint32_t hi[8][2];
    uint32_t lo[F32 ? 8 : 1][2];

    // Requests row `row` (zeros when !ok); finish() turns it into fragments and
    // returns the factor that takes a product with them to the real one.
    __device__ __forceinline__ void request(const void* q, long long row, bool ok, int t) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const long long at = row * kD + Keys::qdim(k >> 1, k & 1, t);
            if constexpr (F32) {
                float2 f = make_float2(0.f, 0.f);
                if (ok) f = __ldg(reinterpret_cast<const float2*>(static_cast<const float*>(q) + at));
                hi[k >> 1][k & 1] = __float_as_uint(f.x);
                lo[k >> 1][k & 1] = __float_as_uint(f.y);
            } else {
                hi[k >> 1][k & 1] = 0u;
                if (ok) hi[k >> 1][k & 1] = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(q) + at));
            }
        }
    }
    __device__ __forceinline__ float finish() {
        if constexpr (F32 || Keys::kF16) {
            float2 f[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                if constexpr (F32)
                    f[k] = make_float2(__uint_as_float(hi[k >> 1][k & 1]), __uint_as_float(lo[k >> 1][k & 1]));
                else
                    f[k] = bf16x2_to_float2(hi[k >> 1][k & 1]);
            }
            // into f16's range: the row's largest value into [2^14, 2^15)
            float mx = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) mx = fmaxf(mx, fmaxf(fabsf(f[k].x), fabsf(f[k].y)));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            float up, down;
            f16_scale(mx, up, down);
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
        } else {
            return 1.f;
        }
    }
    __device__ __forceinline__ float load(const void* q, long long row, bool ok, int t) {
        request(q, row, ok, t);
        return finish();
    }
};

// ---------------------------------------------------------------------------
// ---- equal shares of all keys --------------------------------------------------
// A segment is ROWS rows of one (sequence, kv head); it costs kSegCost and then one
// for every 128 keys that its rows see.  The costs of all segments lie one after the
// other and are cut into equal shares, one per CTA.
constexpr int kUnit = 128;
constexpr int kSegCost = 1;  // query load, merge and store, in units

// The last key that some row of segment rc sees (lo: that every row sees).
template <int ROWS>
__device__ __forceinline__ int last_key(const WalkParams& p, int S, int rc, int* lo = nullptr) {
    if (!p.causal) {
        if (lo) *lo = S - 1;
        return S - 1;
    }
    // rows r0 .. r0 + nrows - 1 are positions r % L
    const int l0 = rc * ROWS % p.L, last = l0 + min(ROWS, p.R - rc * ROWS) - 1;
    if (lo) *lo = (last < p.L ? l0 : 0) + S - p.L;
    return (last < p.L ? last : p.L - 1) + S - p.L;
}
template <int ROWS>
__device__ __forceinline__ int head_cost(const WalkParams& p, int S) {
    if (S == 0) return 0;
    if (!p.causal || p.nrc == 1) return p.nrc * (kSegCost + (S - 1) / kUnit + 1);
    int n = 0;
    for (int rc = 0; rc < p.nrc; ++rc) n += kSegCost + last_key<ROWS>(p, S, rc) / kUnit + 1;
    return n;
}

// share: all costs, cost per share, the sequence that holds the share's first
// position and that sequence's first position.
template <int ROWS>
__device__ __forceinline__ void find_share(const WalkParams& p, int* share) {
    __shared__ int sums[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto cost = [&](int b) { return b < p.B ? p.H_kv * head_cost<ROWS>(p, seq_len(p, b, false)) : 0; };
    const int mine = cost(threadIdx.x);
    int v = mine;
    for (int b = threadIdx.x + kWarps * 32; b < p.B; b += kWarps * 32) v += cost(b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) sums[warp] = v;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += sums[w];
    const int per = max((total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x), p.min_per);
    if (threadIdx.x == 0) {
        share[0] = total;
        share[1] = per;
    }
    const int u = static_cast<int>(blockIdx.x) * per;
    int carry = 0;
    for (int base = 0; base < p.B; base += kWarps * 32) {
        const int b = base + static_cast<int>(threadIdx.x);
        const int x = base == 0 ? mine : cost(b);
        int incl = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        __syncthreads();  // sums is free
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        int before = carry + incl - x;
        for (int w = 0; w < warp; ++w) before += sums[w];
        if (before <= u && u < before + x) {
            share[2] = b;
            share[3] = before;
        }
#pragma unroll
        for (int w = 0; w < kWarps; ++w) carry += sums[w];
    }
    __syncthreads();
}

// Zero rows for the sequences that break the contract, dealt over the CTAs.
template <bool F32>
__device__ __forceinline__ void zero_bad_rows(const WalkParams& p) {
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (seq_len(p, b, threadIdx.x == 0) > 0) continue;
        const long long rows = static_cast<long long>(p.H_kv) * p.R;
        uint4* const o = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + b * rows * kD * (F32 ? 4 : 2));
        for (long long i = threadIdx.x; i < rows * (F32 ? 32 : 16); i += blockDim.x) o[i] = make_uint4(0u, 0u, 0u, 0u);
        if (p.lse)
            for (long long i = threadIdx.x; i < rows; i += blockDim.x) p.lse[b * rows + i] = __int_as_float(0x7f800000);
    }
}

// A piece of a segment: units g0 .. g0 + n - 1 of its ng; unit g lies at position
// seg + kSegCost + g.
template <int ROWS>
struct Segment {
    int b, S, kvh, rc, ng, seg, g0, n;
    __device__ __forceinline__ void cut(const WalkParams& p, int pos, int end) {
        ng = last_key<ROWS>(p, S, rc) / kUnit + 1;
        g0 = max(0, pos - seg - kSegCost);
        n = max(0, min(ng, end - seg - kSegCost) - g0);
    }
    // The first piece with units at or after position pos of sequence b, whose first
    // position is pref; n = 0 if the share ends before one.
    __device__ __forceinline__ void at(const WalkParams& p, int pref, int pos, int end) {
        const int per = head_cost<ROWS>(p, S);
        kvh = (pos - pref) / per;
        seg = pref + kvh * per;
        for (rc = 0;; ++rc) {
            const int c = kSegCost + last_key<ROWS>(p, S, rc) / kUnit + 1;
            if (pos < seg + c) break;
            seg += c;
        }
        cut(p, pos, end);
        if (n == 0) advance(p, end);
    }
    // The next segment's piece; n = 0 past the share.
    __device__ __forceinline__ void advance(const WalkParams& p, int end) {
        seg += kSegCost + ng;
        n = 0;
        if (seg + kSegCost >= end) return;
        if (++rc == p.nrc) {
            rc = 0;
            if (++kvh == p.H_kv) {
                kvh = 0;
                do S = seq_len(p, ++b, false);
                while (S == 0);
            }
        }
        cut(p, seg, end);
    }
    __device__ __forceinline__ bool full() const { return n == ng; }
    // Where the state of an unfinished piece goes: the first slot of the CTA for a
    // segment that began in an earlier share, the second for one that goes on.
    __device__ __forceinline__ long long slot() const { return 2ll * blockIdx.x + (g0 > 0 ? 0 : 1); }
    // The share of the segment's last unit.
    __device__ __forceinline__ int4 crossing(int per) const {
        return make_int4(b, kvh, rc, (seg + kSegCost + ng - 1) / per);
    }
    __device__ __forceinline__ long long row0(const WalkParams& p) const {
        return (static_cast<long long>(b) * p.H_kv + kvh) * p.R + rc * ROWS;
    }
    // The keys of the piece that some row sees end before k1; lo: the last key that
    // every row sees.
    __device__ __forceinline__ void bounds(const WalkParams& p, int& k1, int& lo) const {
        const int hi = last_key<ROWS>(p, S, rc, &lo);
        k1 = S > 0 ? min(hi + 1, (g0 + n) * kUnit) : 0;
    }
};

// The merged row (four dims a lane) and its log-sum-exp.  A sum of 0 is a row without keys;
// one of NaN (a score was NaN; the maximum need not have moved) makes the row NaN.
template <bool F32>
__device__ __forceinline__ void store_row(const WalkParams& p, long long row, int lane, float4 acc, float at, float lt,
                                          float M) {
    const float inv = at == 0.f ? 0.f : 1.f / at;
    if constexpr (F32)
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * kD + 4 * lane) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * kD + 4 * lane) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lane == 0 && p.lse) p.lse[row] = lt == 0.f ? __int_as_float(0x7f800000) : M + log2f(lt);
}

// walk.cu: up to 8 nt rows per CTA (nt = 1, 2; bf16 pages or codes)
struct WalkLaunch {
    int nt;
    bool q4, f32;
    long long items;  // CTAs
    int device;
    cudaStream_t stream;
};
pa_status walk_attend(const WalkParams& p, const WalkLaunch& w);
int walk_resident(int nt, bool q4, bool f32, int rows);  // CTAs per SM
// block.cu: 64 rows per CTA, 2 CTAs per SM
constexpr int kBlockCtaRows = 64;
pa_status block_attend(const WalkParams& p, const WalkLaunch& w);
// Joins the partial states of `shares` CTAs (walk.cu).
pa_status merge_shares(const WalkParams& p, int rows_cta, int shares, bool f32, cudaStream_t stream);
// weights.cu: key weights from stored scores, or from the query, the keys and
// the rows' log-sum-exp (scratch: weights_scratch_bytes, 16-byte aligned).
pa_status weights_from_scores(const WalkParams& p, cudaStream_t stream);
bool weights_supported(const pa_shape& sh, long long w_S, int sm_count);
size_t weights_scratch_bytes(const pa_shape& sh, int sm_count);
size_t weights_scratch_most(const pa_shape& sh, int sm_count);  // ... of any smaller call
pa_status weights_from_keys(const WalkParams& p, bool q4, bool f32, void* scratch, const DeviceInfo& dev,
                            cudaStream_t stream);
// The query rows of a (sequence, kv head) cut into n runs, each CTA taking one; n > 1:
// their sums in part, [run][(b, kvh)][key < max_S].
struct RowSplits {
    float* part;
    int n;
    __device__ __forceinline__ float* at(const WalkParams& p, int run, int bk) const {
        return part + (static_cast<long long>(run) * p.B * p.H_kv + bk) * p.max_S;
    }
};
// weights_tiles.cu: the same for bf16 queries on tcgen05 (n up to ceil(R / 64))
pa_status weights_on_tiles(const WalkParams& p, bool q4, const RowSplits& sp, const DeviceInfo& dev,
                           cudaStream_t stream);

}  // namespace walk
}  // namespace pa
