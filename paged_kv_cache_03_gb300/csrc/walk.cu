// walk.cu -- attention over 4-bit pages, and attention that also accumulates
// each key's weight, over 4-bit or bf16 pages.
//
// For a (sequence, kv head) with rows r = (query head of the group, position)
//   s[r][k] = scale * q_r . K_k  (k <= position's frontier),
//   out_r = sum_k softmax(s_r)[k] V_k,   w_out[k] = w_in[k] + sum_r softmax(s_r)[k].
//
// Layout.  A segment is up to 8 * NT rows of one (sequence, kv head).  The keys
// of all segments, in units of 128, are cut into equal shares, one per resident
// CTA (four warps); in each segment of its share a warp takes every fourth step
// of 32 keys (16 over bf16 pages) with its own running max, sum and O, and the
// warps merge at the end.  Segments that cross shares leave partial states, which
// walk_combine_kernel merges.  Equal shares keep ragged batches balanced and pay
// the start of a pipeline once per CTA.
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
    // partial states: max, sum of the applied weights, sum; O.  walk_kernel: two
    // slots per CTA of its rows; block_kernel: [(b, kvh, row)][chunk]
    float4* part_ml;
    float* part_o;
    float* lse;       // [(b, kvh, row)] log2 of the sum of 2^score, or null
    float* score;     // [(b, kvh)][key < cap][row] scores in log2 units, or null
    long long cap;    // keys of a (b, kvh) in score
    const float* w_in;
    float* w_out;
    long long w_S;
    uint32_t* flag;
    int B, H_kv, L, R, num_pages, ps, max_npg, causal, nrc;
    int nkc, C;   // block_kernel: key chunks of a row, keys per chunk
    int whole;    // walk_kernel: 1 one CTA per segment, 0 equal shares of all keys
    int min_per;  // least units of a share
    int* prefix;  // [B] first unit of a sequence, [B] all units, [B + 1] units per share
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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(ok ? 8 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
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

template <bool F16>
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        mma_16816_f16_first(d, a, b0, b1);
    else
        mma_16816_bf16_first(d, a, b0, b1);
}
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        mma_16816_f16(d, a, b0, b1);
    else
        mma_16816_bf16(d, a, b0, b1);
}

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
        if constexpr (!F32 && !Keys::kF16) return 1.f;
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
    }
    __device__ __forceinline__ float load(const void* q, long long row, bool ok, int t) {
        request(q, row, ok, t);
        return finish();
    }
};

// ---------------------------------------------------------------------------
// Units of 128 keys (a step of every warp, or two) are what the shares count.
constexpr int kUnit = 128;

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// This CTA's equal share of the keys of all segments (sequence, kv head, row
// chunk): share = all units, units per share, the sequence that holds the
// share's first unit and that sequence's first unit.  CTA 0 also leaves the
// sequences' first units in p.prefix for the merge.
__device__ __forceinline__ void find_share(const WalkParams& p, int* share) {
    __shared__ int sums[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int segs = p.H_kv * p.nrc;
    auto units = [&](int b) { return b < p.B ? (seq_len(p, b, false) + kUnit - 1) / kUnit * segs : 0; };
    const int mine = units(threadIdx.x);
    int v = mine;
    for (int b = threadIdx.x + kWarps * 32; b < p.B; b += kWarps * 32) v += units(b);
    v = warp_sum(v);
    if (lane == 0) sums[warp] = v;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += sums[w];
    const int per = max((total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x), p.min_per);
    if (threadIdx.x == 0) {
        share[0] = total;
        share[1] = per;
        if (blockIdx.x == 0) {
            p.prefix[p.B] = total;
            p.prefix[p.B + 1] = per;
        }
    }
    const int u = static_cast<int>(blockIdx.x) * per;
    int carry = 0;
    for (int base = 0; base < p.B; base += kWarps * 32) {
        const int b = base + static_cast<int>(threadIdx.x);
        const int x = base == 0 ? mine : units(b);
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
        if (b < p.B) {
            if (blockIdx.x == 0) p.prefix[b] = before;
            if (before <= u && u < before + x) {
                share[2] = b;
                share[3] = before;
            }
        }
#pragma unroll
        for (int w = 0; w < kWarps; ++w) carry += sums[w];
    }
    __syncthreads();
}

// A piece of a segment: units g0 .. g0 + n - 1 of its ng.
struct Segment {
    int b, S, pref;  // sequence, its length and first unit
    int kvh, rc, ng, g0, n;
    // The piece at unit `pos` of sequence b (which has it), up to unit `end`.
    __device__ __forceinline__ void at(const WalkParams& p, int pos, int end) {
        ng = (S + kUnit - 1) / kUnit;
        const int sib = (pos - pref) / ng;
        g0 = (pos - pref) - sib * ng;
        kvh = sib / p.nrc;
        rc = sib - kvh * p.nrc;
        n = min(ng - g0, end - pos);
    }
    // On to unit `pos`, the one after this piece.
    __device__ __forceinline__ void advance(const WalkParams& p, int pos, int end) {
        if (pos == pref + ng * p.H_kv * p.nrc) {  // the next sequence with keys
            pref = pos;
            do S = seq_len(p, ++b, false);
            while (S == 0);
        }
        at(p, pos, end);
    }
    __device__ __forceinline__ long long row0(const WalkParams& p, int rows) const {
        return (static_cast<long long>(b) * p.H_kv + kvh) * p.R + rc * rows;
    }
    // k1: the keys of the piece that some row sees end before it; lo: the last key
    // that every row sees.
    template <int ROWS>
    __device__ __forceinline__ void bounds(const WalkParams& p, int& k1, int& lo) const {
        int hi = S - 1;
        lo = hi;
        if (p.causal) {  // rows r0 .. r0 + nrows - 1 are positions r % L
            const int l0 = rc * ROWS % p.L, last = l0 + min(ROWS, p.R - rc * ROWS) - 1;
            hi = (last < p.L ? last : p.L - 1) + S - p.L;
            lo = (last < p.L ? l0 : 0) + S - p.L;
        }
        k1 = S > 0 ? min(hi + 1, (g0 + n) * kUnit) : 0;
    }
};

// The merged row (four dims a lane) and its log-sum-exp.
template <bool F32>
__device__ __forceinline__ void store_row(const WalkParams& p, long long row, int lane, float4 acc, float at, float lt,
                                          float M) {
    const float inv = at > 0.f ? 1.f / at : 0.f;
    if constexpr (F32)
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * kD + 4 * lane) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * kD + 4 * lane) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lane == 0 && p.lse) p.lse[row] = lt > 0.f ? M + log2f(lt) : __int_as_float(0x7f800000);
}

// CTAs of walk_kernel resident per SM.
constexpr int resident_ctas(int nt, bool q4, bool f32) { return nt == 2 ? 2 : f32 || !q4 ? 3 : 4; }
constexpr size_t walk_smem(bool q4, int rows) {
    return kWarps * 2 * (q4 ? Stage<true>::kBytes : Stage<false>::kBytes) + sizeof(float) * kWarps * rows * kMerge;
}

template <class Keys, class Values, int NT, bool F32, bool A16, bool W>
__global__ void __launch_bounds__(kWarps * 32, resident_ctas(NT, Keys::kF16, F32)) walk_kernel(const WalkParams p) {
    constexpr bool F16 = Keys::kF16;
    constexpr int ROWS = 8 * NT;
    constexpr int U = Keys::kU, kStep = 16 * U;
    using St = Stage<F16>;
    extern __shared__ __align__(1024) uint8_t smem[];  // the warps' stages, then the merge buffer:
    const int mrows = min(ROWS, p.R);                  // [warp][row][kMerge]: o, max, applied sum, sum
    float* const merge = reinterpret_cast<float*>(smem + kWarps * 2 * St::kBytes);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    __shared__ int share[4];  // total units, units per share, first sequence, its first unit
    pdl_launch_dependents();
    Segment sg;
    int pos = 0, end = 0;  // units of this CTA's share
    if (p.whole) {
        int item = static_cast<int>(blockIdx.x);
        sg.rc = item % p.nrc;
        item /= p.nrc;
        sg.kvh = item % p.H_kv;
        sg.b = item / p.H_kv;
        sg.S = seq_len(p, sg.b, sg.rc == 0 && sg.kvh == 0 && threadIdx.x == 0);
        sg.pref = sg.g0 = 0;
        sg.ng = sg.n = (sg.S + kUnit - 1) / kUnit;
    } else {
        find_share(p, share);
        pos = static_cast<int>(blockIdx.x) * share[1];
        end = min(pos + share[1], share[0]);
        if (pos >= end) return;
        sg.b = share[2];
        sg.pref = share[3];
        sg.S = seq_len(p, sg.b, false);
        sg.at(p, pos, end);
    }
    const uint32_t ring = smem_u32(smem) + warp * 2 * St::kBytes;
    uint32_t st = ring;
    StepWalker<A16, U> wk;
    int pg[2] = {-1, -1};
    QueryFrags<Keys, F32> q[NT];
    // Requests the first stage, the page ids after it and the query rows of `sg`.
    auto open_keys = [&]() {
        int k1, lo;
        sg.bounds<ROWS>(p, k1, lo);
        const int first = sg.g0 * kUnit + warp * kStep;
        wk.start(p, A16 ? first : first + lane, kWarps * kStep);
        const int npg = (sg.S + p.ps - 1) / p.ps;
        const int32_t* const table = p.bt + static_cast<long long>(sg.b) * p.max_npg;
        wk.pages(table, p, first < k1 ? npg : 0, pg);
        St::fill(p, wk.rows(p, sg.kvh, pg), st, lane);
        wk.next(p);
        wk.pages(table, p, first + kWarps * kStep < k1 ? npg : 0, pg);
        cp_async_commit();
    };
    auto open_query = [&]() {
        const long long row0 = sg.row0(p, ROWS);
#pragma unroll
        for (int n = 0; n < NT; ++n) q[n].request(p.q, row0 + 8 * n + g, sg.rc * ROWS + 8 * n + g < p.R, t);
    };
    open_query();
    open_keys();

    for (;;) {  // segments of the share
    const int S = sg.S, b = sg.b, kvh = sg.kvh;
    const int r0 = sg.rc * ROWS, nrows = min(ROWS, p.R - r0);
    const long long row0 = sg.row0(p, ROWS);
    const int npg = (S + p.ps - 1) / p.ps;
    const int32_t* const table = p.bt + static_cast<long long>(b) * p.max_npg;
    int k1, lim_min;  // last key any row sees + 1 (within the share), last key every row sees
    sg.bounds<ROWS>(p, k1, lim_min);
    // the last key each of this lane's rows (2t, 2t + 1 of every n-tile) sees
    int lim[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int rr = 8 * n + 2 * t + e;
            lim[n][e] = rr < nrows ? (p.causal ? (r0 + rr) % p.L + S - p.L : S - 1) : -1;
        }
    float qs[NT][2];  // score scale of rows 2t, 2t + 1 in log2 units
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const float down = q[n].finish();
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

    // Each warp has two stages of its own: the next step is requested when a
    // step begins, the next segment's first one when a segment's last step ends.
    for (int base = sg.g0 * kUnit + warp * kStep; base < k1; base += kWarps * kStep) {
        __syncwarp();  // the other stage has been read
        const uint32_t st_next = st == ring ? ring + St::kBytes : ring;
        St::fill(p, wk.rows(p, kvh, pg), st_next, lane);  // (zeros past the last step: no branch)
        wk.next(p);
        wk.pages(table, p, base + 2 * kWarps * kStep < k1 ? npg : 0, pg);
        cp_async_commit();
        cp_async_wait<1>();
        __syncwarp();
        Keys kk[U];
#pragma unroll
        for (int u = 0; u < U; ++u) kk[u].load(st, u, g, t);
        // S^T: 16 U keys x 8 NT rows
        float s[NT][U][4];
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
                        if (i == 0 && j == 0)
                            mma_first<F16>(s[n][u], a[j], q[n].hi[0][0], q[n].hi[0][1]);
                        else
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
        if constexpr (W) {  // (keys past the chunk's last one stay inside the table)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int key = base + 16 * u + g + 8 * h, rr = 8 * n + 2 * t;
                        if (key >= p.cap) continue;
                        float* const to = p.score + ((static_cast<long long>(b) * p.H_kv + kvh) * p.cap + key) * p.R + rr;
                        const float x0 = s[n][u][2 * h] * qs[n][0], x1 = s[n][u][2 * h + 1] * qs[n][1];
                        if (rr + 1 < nrows && p.R % 2 == 0) {
                            *reinterpret_cast<float2*>(to) = make_float2(x0, x1);
                        } else {
                            if (rr < nrows) to[0] = x0;
                            if (rr + 1 < nrows) to[1] = x1;
                        }
                    }
        }
        uint32_t pb[NT][U][2], pl[NT][U][2];  // P^T fragments, and their low parts
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float mt[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
                mt[e] = fmax3(fmaxf(s[n][0][e], s[n][0][2 + e]), s[n][U - 1][e], s[n][U - 1][2 + e]) * qs[n][e];
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
        Values vv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) vv[u].load(st, u, g, t);
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
        st = st_next;
    }
    const Segment done = sg;
    pos += sg.n;
    const bool more = pos < end;
    if (more) {
        sg.advance(p, pos, end);
        cp_async_wait<0>();  // the last step's empty fill of the same stage
        __syncwarp();
        open_keys();
    }

    // ---- merge the four warps ---------------------------------------------
    float* const mw = merge + warp * mrows * kMerge;
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
            if (8 * n + 2 * t + e >= mrows) continue;
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
    if (more) open_query();
    __syncthreads();
    const bool full = done.n == done.ng;
    for (int rr = warp; rr < nrows; rr += kWarps) {  // a warp per row, four dims a lane
        const float* const mr = merge + rr * kMerge;
        float mv[kWarps], M = neg_inf();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            mv[w] = mr[w * mrows * kMerge + kD];
            M = fmaxf(M, mv[w]);
        }
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float at = 0.f, lt = 0.f;
        if (M != neg_inf()) {
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float* const mw_ = mr + w * mrows * kMerge;
                const float a = fast_exp2(mv[w] - M);
                const float4 x = *reinterpret_cast<const float4*>(mw_ + 4 * lane);
                acc.x += a * x.x;
                acc.y += a * x.y;
                acc.z += a * x.z;
                acc.w += a * x.w;
                at += a * mw_[kD + 1];
                lt += a * mw_[kD + 2];
            }
        }
        if (full) {
            store_row<F32>(p, row0 + rr, lane, acc, at, lt, M);
        } else {
            // a share's segment that began in an earlier one, or its last one
            const long long row = static_cast<long long>(2 * blockIdx.x + (done.g0 > 0 ? 0 : 1)) * ROWS + rr;
            if (lane == 0) p.part_ml[row] = make_float4(M, at, lt, 0.f);
            if (M != neg_inf()) *reinterpret_cast<float4*>(p.part_o + row * kD + 4 * lane) = acc;
        }
    }
    if (!more) break;
    __syncthreads();  // the merge buffer is free
    }
    cp_async_wait<0>();
    report_pages(p, wk.bad);
}

// Merges the pieces of a segment that several shares hold: one CTA per row, its
// warps take every fourth piece, four dims a lane.  Rows of sequences that
// break the contract are written as zeros.
template <bool F32>
__global__ void __launch_bounds__(kWarps * 32) walk_combine_kernel(const WalkParams p, int rows_cta) {
    __shared__ float4 mls[kWarps];
    __shared__ float4 os[kWarps][32];
    pdl_launch_dependents();
    pdl_wait_primary();
    const int per_seg = min(rows_cta, p.R);
    const int seg = static_cast<int>(blockIdx.x) / per_seg, rr = static_cast<int>(blockIdx.x) - seg * per_seg;
    const int bk = seg / p.nrc, rc = seg - bk * p.nrc;
    const int b = bk / p.H_kv, kvh = bk - b * p.H_kv;
    if (rc * rows_cta + rr >= p.R) return;
    const long long row = static_cast<long long>(bk) * p.R + rc * rows_cta + rr;
    const int S = seq_len(p, b, kvh == 0 && rc == 0 && rr == 0 && threadIdx.x == 0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ng = (S + kUnit - 1) / kUnit, per = p.prefix[p.B + 1];
    const int first = p.prefix[b] + (kvh * p.nrc + rc) * ng;
    const int c0 = first / per, c1 = ng > 0 ? (first + ng - 1) / per : c0 - 1;
    if (c0 == c1) return;  // one share wrote it
    // slot of piece i: the first share's last segment, then the others' first
    auto slot = [&](int i) { return static_cast<long long>(i == 0 ? 2 * c0 + 1 : 2 * (c0 + i)) * rows_cta + rr; };
    const int np = c1 - c0 + 1;
    float M = neg_inf(), at = 0.f, lt = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int base = 0; base < np; base += 32 * kWarps) {  // lane i: piece base + 4 i + warp
        const int mine = base + kWarps * lane + warp;
        const float4 v = mine < np ? p.part_ml[slot(mine)] : make_float4(neg_inf(), 0.f, 0.f, 0.f);
        float mt = v.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
        if (mt == neg_inf()) continue;
        if (mt > M) {
            const float a = fast_exp2(M - mt);  // 2^-inf = 0 at the start
            acc.x *= a;
            acc.y *= a;
            acc.z *= a;
            acc.w *= a;
            at *= a;
            lt *= a;
            M = mt;
        }
        const float mine_a = fast_exp2(v.x - M);  // 0 for a piece without keys
        const int n = min(32, (np - base - warp + kWarps - 1) / kWarps);
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const float a = __shfl_sync(0xffffffffu, mine_a, i);
            const float y = __shfl_sync(0xffffffffu, v.y, i), z = __shfl_sync(0xffffffffu, v.z, i);
            if (a == 0.f) continue;  // (its O was not written)
            const float4 x = *reinterpret_cast<const float4*>(p.part_o + slot(base + kWarps * i + warp) * kD + 4 * lane);
            at += a * y;
            lt += a * z;
            acc.x += a * x.x;
            acc.y += a * x.y;
            acc.z += a * x.z;
            acc.w += a * x.w;
        }
    }
    if (lane == 0) mls[warp] = make_float4(M, at, lt, 0.f);
    os[warp][lane] = acc;
    __syncthreads();
    if (warp > 0) return;
    float Mx = neg_inf();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) Mx = fmaxf(Mx, mls[w].x);
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    at = lt = 0.f;
    if (Mx != neg_inf()) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float a = fast_exp2(mls[w].x - Mx);
            const float4 x = os[w][lane];
            at += a * mls[w].y;
            lt += a * mls[w].z;
            acc.x += a * x.x;
            acc.y += a * x.y;
            acc.z += a * x.z;
            acc.w += a * x.w;
        }
    }
    store_row<F32>(p, row, lane, acc, at, lt, Mx);
}

// Merges the key chunks of a row: one warp per row, four dims per lane.  A
// row without keys is written as zeros.
template <bool F32>
__global__ void __launch_bounds__(128) block_combine_kernel(const WalkParams p) {
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
    store_row<F32>(p, row, lane, acc, at, lt, M);
}

// ---- many rows: tiles of 64 keys shared by 64 rows --------------------------
//
// With more rows than a warp holds, dequantising per warp would cost more than
// the products.  Here a CTA's four warps take 16 rows each (M = rows) and the
// 64-key K and V tiles go through shared memory once, as f16 (4-bit pages) or
// as they are (bf16): S = Q K^T with K by ldmatrix, O += P V with V by
// ldmatrix.trans.  Two buffers: the next tile is requested when a tile begins
// and, 4-bit, written dequantised when it ends.  A 256-byte row holds its even
// 16-byte chunks first, then the odd ones, both permuted by the row's low bits:
// the writers (32 bytes a lane) and ldmatrix meet no bank conflict.
constexpr int kTK = 64;
constexpr int kTileBytes = kTK * kD * 2;

__device__ __forceinline__ uint32_t chunk_at(int row, int c) {
    return static_cast<uint32_t>(row * 256 + (c & 1) * 128 + (((c >> 1) ^ (row & 7)) << 4));
}

template <bool Q4>
struct TileLoader;

template <>
struct TileLoader<true> {  // thread: dims 16 grp .. of keys (tid >> 3) + 16 i
    bool bad = false;
    uint2 c[4][2];
    uint32_t s[4][2];
    __device__ __forceinline__ void request(const WalkParams& p, int b, int kvh, int base, int S, uint32_t, uint32_t) {
        const int grp = threadIdx.x & 7;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int key = base + static_cast<int>(threadIdx.x >> 3) + 16 * i;
            const int lp = key / p.ps;
            const int pg = key < S ? __ldg(p.bt + static_cast<long long>(b) * p.max_npg + lp) : kNoPage;
            const long long r = row_in(p, kvh, pg, key - lp * p.ps, bad);
            c[i][0] = c[i][1] = make_uint2(0u, 0u);
            s[i][0] = s[i][1] = 0u;
            if (r >= 0) {
                c[i][0] = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.kc) + r * kQ4CodeBytes) + grp);
                c[i][1] = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.vc) + r * kQ4CodeBytes) + grp);
                s[i][0] = __ldg(static_cast<const uint8_t*>(p.ks) + r * kQ4Groups + grp);
                s[i][1] = __ldg(static_cast<const uint8_t*>(p.vs) + r * kQ4Groups + grp);
            }
        }
    }
    __device__ __forceinline__ void finish(uint32_t kbuf, uint32_t vbuf) {
        const int grp = threadIdx.x & 7;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = static_cast<int>(threadIdx.x >> 3) + 16 * i;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const uint32_t s2 = e4m3x2_to_f16x2(s[i][kv] | (s[i][kv] << 8));
                uint32_t h[8];
                e2m1x8_to_f16x2(c[i][kv].x, *reinterpret_cast<uint32_t(*)[4]>(h));
                e2m1x8_to_f16x2(c[i][kv].y, *reinterpret_cast<uint32_t(*)[4]>(h + 4));
#pragma unroll
                for (int j = 0; j < 8; ++j) h[j] = hmul2(h[j], s2);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"((kv ? vbuf : kbuf) + chunk_at(row, 2 * grp + j)),
                                 "r"(h[4 * j]), "r"(h[4 * j + 1]), "r"(h[4 * j + 2]), "r"(h[4 * j + 3])
                                 : "memory");
            }
        }
    }
};

template <>
struct TileLoader<false> {  // thread: chunk tid & 15 of keys (tid >> 4) + 8 i
    bool bad = false;
    __device__ __forceinline__ void request(const WalkParams& p, int b, int kvh, int base, int S, uint32_t kbuf,
                                            uint32_t vbuf) {
        const int c = threadIdx.x & 15;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = static_cast<int>(threadIdx.x >> 4) + 8 * i, key = base + row;
            const int lp = key / p.ps;
            const int pg = key < S ? __ldg(p.bt + static_cast<long long>(b) * p.max_npg + lp) : kNoPage;
            const int r = row_in(p, kvh, pg, key - lp * p.ps, bad);
            const long long off = r >= 0 ? static_cast<long long>(r) * (2 * kD) + 16 * c : 0;
            cp_async16(kbuf + chunk_at(row, c), static_cast<const uint8_t*>(p.kc) + off, r >= 0);
            cp_async16(vbuf + chunk_at(row, c), static_cast<const uint8_t*>(p.vc) + off, r >= 0);
        }
        cp_async_commit();
    }
    __device__ __forceinline__ void finish(uint32_t, uint32_t) { cp_async_wait<0>(); }
};

// Dim pairs of Q's A fragments: the natural order (K's tile is in it).
template <bool Q4>
struct NaturalDims {
    static constexpr bool kF16 = Q4;
    __device__ static int qdim(int j, int half, int t) { return 16 * j + 8 * half + 2 * t; }
};

template <bool Q4, bool F32>
__global__ void __launch_bounds__(kWarps * 32) block_kernel(const WalkParams p) {
    constexpr int ROWS = 16 * kWarps;
    extern __shared__ __align__(1024) uint8_t smem[];  // K, V, K, V tiles
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    int item = static_cast<int>(blockIdx.x);
    const int kc = item % p.nkc;
    item /= p.nkc;
    const int rc = p.nrc - 1 - item % p.nrc;  // the longest rows first
    item /= p.nrc;
    const int kvh = item % p.H_kv, b = item / p.H_kv;
    const int S = seq_len(p, b, kc == 0 && rc == 0 && kvh == 0 && threadIdx.x == 0);
    const int r0 = rc * ROWS, nrows = min(ROWS, p.R - r0);
    const long long row0 = (static_cast<long long>(b) * p.H_kv + kvh) * p.R + r0;
    // the last key each of this lane's rows (g, g + 8 of the warp's 16) sees, and
    // the extremes over the warp and the CTA
    int lim[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int rr = 16 * warp + g + 8 * e;
        lim[e] = rr < nrows ? (p.causal ? (r0 + rr) % p.L + S - p.L : S - 1) : -1;
    }
    int cta_max = S - 1;
    if (p.causal) {  // rows r0 .. r0 + nrows - 1: positions r % L
        const int l0 = r0 % p.L;
        cta_max = (l0 + nrows - 1 >= p.L ? p.L - 1 : l0 + nrows - 1) + S - p.L;
    }
    int lim_min = min(lim[0] < 0 ? INT_MAX : lim[0], lim[1] < 0 ? INT_MAX : lim[1]), lim_max = max(lim[0], lim[1]);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, o));
        lim_max = max(lim_max, __shfl_xor_sync(0xffffffffu, lim_max, o));
    }
    const int k0 = kc * p.C, k1 = S > 0 ? min(cta_max + 1, k0 + p.C) : 0;

    // A fragments of the warp's 16 rows: two sets of 8 rows, as B fragments are
    QueryFrags<NaturalDims<Q4>, F32> q[2];
    float qs[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int rr = 16 * warp + g + 8 * e;
        qs[e] = fmaxf(q[e].load(p.q, row0 + rr, rr < nrows, t) * p.scale_log2, FLT_MIN);
    }
    float m[2] = {neg_inf(), neg_inf()}, l[2] = {0.f, 0.f}, la[2] = {0.f, 0.f};
    float o[16][4];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    const uint32_t buf = smem_u32(smem);
    TileLoader<Q4> ld;
    if (k0 < k1) {
        ld.request(p, b, kvh, k0, S, buf, buf + kTileBytes);
        ld.finish(buf, buf + kTileBytes);
    }
    int cur = 0;
    for (int base = k0; base < k1; base += kTK, cur ^= 1) {
        __syncthreads();  // the tile is whole; the other buffer is no longer read
        const uint32_t kb = buf + cur * 2 * kTileBytes, vb = kb + kTileBytes;
        const uint32_t kn = buf + (cur ^ 1) * 2 * kTileBytes, vn = kn + kTileBytes;
        const bool more = base + kTK < k1;
        if (more) ld.request(p, b, kvh, base + kTK, S, kn, vn);
        if (base <= lim_max) {  // (uniform over the warp)
            float s[8][4];
#pragma unroll
            for (int n = 0; n < 8; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {  // 16 dims
                const uint32_t a[4] = {q[0].hi[j][0], q[1].hi[j][0], q[0].hi[j][1], q[1].hi[j][1]};
                uint32_t al[4];
                if constexpr (F32) {
                    al[0] = q[0].lo[j][0];
                    al[1] = q[1].lo[j][0];
                    al[2] = q[0].lo[j][1];
                    al[3] = q[1].lo[j][1];
                }
#pragma unroll
                for (int n = 0; n < 8; n += 2) {  // 16 keys
                    uint32_t x[4];
                    ldmatrix_x4(x, kb + chunk_at(8 * n + (lane & 7) + 8 * (lane >> 4), 2 * j + ((lane >> 3) & 1)));
                    mma<Q4>(s[n], a, x[0], x[1]);
                    mma<Q4>(s[n + 1], a, x[2], x[3]);
                    if constexpr (F32) {
                        mma<Q4>(s[n], al, x[0], x[1]);
                        mma<Q4>(s[n + 1], al, x[2], x[3]);
                    }
                }
            }
            if (base + kTK - 1 > lim_min) {
#pragma unroll
                for (int n = 0; n < 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (base + 8 * n + 2 * t + (e & 1) > lim[e >> 1]) s[n][e] = neg_inf();
            }
            float mt[2] = {neg_inf(), neg_inf()};
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                mt[0] = fmax3(mt[0], s[n][0], s[n][1]);
                mt[1] = fmax3(mt[1], s[n][2], s[n][3]);
            }
            mt[0] *= qs[0];
            mt[1] *= qs[1];
            if (__any_sync(0xffffffffu, mt[0] > m[0] + kLazyRescaleLog2 || mt[1] > m[1] + kLazyRescaleLog2)) {
                float al[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mt[e] = fmaxf(mt[e], __shfl_xor_sync(0xffffffffu, mt[e], 1));
                    mt[e] = fmaxf(mt[e], __shfl_xor_sync(0xffffffffu, mt[e], 2));
                    const bool grow = mt[e] > m[e] + kLazyRescaleLog2;
                    al[e] = grow ? fast_exp2(m[e] - mt[e]) : 1.f;  // 2^-inf = 0 at the start
                    if (grow) m[e] = mt[e];
                    l[e] *= al[e];
                    la[e] *= al[e];
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    o[i][0] *= al[0];
                    o[i][1] *= al[0];
                    o[i][2] *= al[1];
                    o[i][3] *= al[1];
                }
            }
            const float mu[2] = {m[0] == neg_inf() ? 0.f : m[0], m[1] == neg_inf() ? 0.f : m[1]};
#pragma unroll
            for (int n = 0; n < 8; n += 2) {  // 16 keys: P's A fragment, then O += P V
                uint32_t a[4], al[4];
#pragma unroll
                for (int h = 0; h < 2; ++h)  // keys 8 (n + h) .., rows g and g + 8
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float p0 = fast_exp2(fmaf(s[n + h][2 * e], qs[e], -mu[e]));
                        const float p1 = fast_exp2(fmaf(s[n + h][2 * e + 1], qs[e], -mu[e]));
                        l[e] += p0 + p1;
                        if constexpr (Q4) {
                            const uint32_t x = pack_f16x2(p0, p1);
                            a[2 * h + e] = x;
                            if constexpr (F32) {
                                const float2 f = f16x2_to_float2(x);
                                al[2 * h + e] = pack_f16x2(p0 - f.x, p1 - f.y);
                            }
                        } else {
                            const uint32_t x = pack_bf16x2(p0, p1);
                            const float2 f = bf16x2_to_float2(x);
                            la[e] += f.x + f.y;
                            a[2 * h + e] = x;
                        }
                    }
#pragma unroll
                for (int d = 0; d < 16; d += 2) {  // 16 dims
                    uint32_t x[4];
                    ldmatrix_x4_trans(x, vb + chunk_at(8 * n + (lane & 15), d + (lane >> 4)));
                    mma<Q4>(o[d], a, x[0], x[1]);
                    mma<Q4>(o[d + 1], a, x[2], x[3]);
                    if constexpr (F32) {
                        mma<Q4>(o[d], al, x[0], x[1]);
                        mma<Q4>(o[d + 1], al, x[2], x[3]);
                    }
                }
            }
        }
        if (more) ld.finish(kn, vn);
    }
    report_pages(p, ld.bad);
    // rows g and g + 8: dims 8 d + 2t, + 1
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], d);
            la[e] += __shfl_xor_sync(0xffffffffu, la[e], d);
        }
        const int rr = 16 * warp + g + 8 * e;
        if (rr >= nrows) continue;
        const float at = Q4 ? l[e] : la[e];
        const long long row = row0 + rr;
        if (p.nkc == 1) {
            const float inv = at > 0.f ? 1.f / at : 0.f;
#pragma unroll
            for (int d = 0; d < 16; ++d) {
                const float x = o[d][2 * e] * inv, y = o[d][2 * e + 1] * inv;
                if constexpr (F32)
                    *reinterpret_cast<float2*>(static_cast<float*>(p.out) + row * kD + 8 * d + 2 * t) = make_float2(x, y);
                else
                    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + row * kD + 8 * d + 2 * t) = pack_bf16x2(x, y);
            }
            if (t == 0 && p.lse) p.lse[row] = l[e] > 0.f ? m[e] + log2f(l[e]) : __int_as_float(0x7f800000);
        } else {
            if (t == 0) p.part_ml[row * p.nkc + kc] = make_float4(l[e] > 0.f ? m[e] : neg_inf(), at, l[e], 0.f);
            if (l[e] > 0.f) {
#pragma unroll
                for (int d = 0; d < 16; ++d)
                    *reinterpret_cast<float2*>(p.part_o + (row * p.nkc + kc) * kD + 8 * d + 2 * t) =
                        make_float2(o[d][2 * e], o[d][2 * e + 1]);
            }
        }
    }
}

// w_out[b, kvh, k] = w_in[b, kvh, k] + the rows' probabilities of key k, 0 past
// the context, from the scores that walk_kernel left.  One thread per key; the
// R scores of a key lie together, so a warp reads them as whole lines.
__global__ void __launch_bounds__(256) walk_sum_kernel(const WalkParams p, int ntile) {
    pdl_wait_primary();
    const int tile = static_cast<int>(blockIdx.x) % ntile;
    const long long bk = static_cast<int>(blockIdx.x) / ntile;
    const long long k = static_cast<long long>(tile) * 256 + threadIdx.x;
    if (k >= p.w_S) return;
    const int S = seq_len(p, static_cast<int>(bk / p.H_kv), false);
    float acc = 0.f;
    if (k < S) {
        const float* const x = p.score + (bk * p.cap + k) * p.R;
        const float* const lse = p.lse + bk * p.R;
        if (p.R % 4 == 0) {
            for (int r = 0; r < p.R; r += 4) {
                const float4 v = *reinterpret_cast<const float4*>(x + r);
                acc += fast_exp2(v.x - lse[r]);
                acc += fast_exp2(v.y - lse[r + 1]);
                acc += fast_exp2(v.z - lse[r + 2]);
                acc += fast_exp2(v.w - lse[r + 3]);
            }
        } else {
            for (int r = 0; r < p.R; ++r) acc += fast_exp2(x[r] - lse[r]);
        }
        if (p.w_in) acc += p.w_in[bk * p.w_S + k];
    }
    p.w_out[bk * p.w_S + k] = acc;
}

// The same from the query and the keys, for many rows: a CTA takes 128 keys of
// one (sequence, kv head), each warp 32 of them as A fragments in registers, and
// runs over the rows in chunks of 64 whose B fragments the warps lay out in
// shared memory once per chunk (16 bytes a lane and k-step pair).  Bound by the
// warp-level MMA rate (8 cycles per m16n8k16 and SM sub-partition).
constexpr int kChunkTiles = 8;  // n-tiles of 8 rows per shared-memory chunk

template <class Keys, bool F32>
__global__ void __launch_bounds__(kWarps * 32) walk_weights_kernel(const WalkParams p, int ntile) {
    constexpr int PARTS = F32 ? 2 : 1;
    __shared__ uint4 qsm[PARTS][kChunkTiles][4][32];
    __shared__ float qs_s[kChunkTiles * 8], lse_s[kChunkTiles * 8];
    __shared__ int lim_s[kChunkTiles * 8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int tile = static_cast<int>(blockIdx.x) % ntile, bk = static_cast<int>(blockIdx.x) / ntile;
    const int b = bk / p.H_kv, kvh = bk - b * p.H_kv;
    const long long cta0 = static_cast<long long>(tile) * (32 * kWarps);
    const int S = seq_len(p, b, false);
    float acc[2][2] = {};  // keys g and g + 8 of both halves, this lane's rows
    if (cta0 < S) {        // (uniform over the CTA)
        const int k0 = static_cast<int>(cta0) + 32 * warp;
        uint32_t a[2][8][4];
        {
            StepWalker<false, 2> wk;
            wk.start(p, k0 + lane, 0);
            int pg[2];
            wk.pages(p.bt + static_cast<long long>(b) * p.max_npg, p, k0 + lane < S ? INT_MAX : 0, pg);
            const StepRows<false, 2> rows = wk.rows(p, kvh, pg);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                Keys kk;
                kk.load(p, rows, u, g, t);
                const typename Keys::Scales ksc = kk.scales();
#pragma unroll
                for (int i = 0; i < 4; ++i) kk.frags(ksc, i, *reinterpret_cast<uint32_t(*)[2][4]>(a[u][2 * i]));
            }
        }
        const long long row0 = static_cast<long long>(bk) * p.R;
        for (int r0 = 0; r0 < p.R; r0 += 8 * kChunkTiles) {
            const int nt = min(kChunkTiles, (p.R - r0 + 7) / 8);
            __syncthreads();
            for (int n = warp; n < nt; n += kWarps) {
                const int r = r0 + 8 * n + g;
                QueryFrags<Keys, F32> q;
                const float down = q.load(p.q, row0 + r, r < p.R, t);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    qsm[0][n][i][lane] = make_uint4(q.hi[2 * i][0], q.hi[2 * i][1], q.hi[2 * i + 1][0], q.hi[2 * i + 1][1]);
                    if constexpr (F32)
                        qsm[1][n][i][lane] = make_uint4(q.lo[2 * i][0], q.lo[2 * i][1], q.lo[2 * i + 1][0], q.lo[2 * i + 1][1]);
                }
                if (t == 0) {
                    qs_s[8 * n + g] = fmaxf(down * p.scale_log2, FLT_MIN);
                    // (a row past the last one weighs 2^-inf = 0)
                    lse_s[8 * n + g] = r < p.R ? p.lse[row0 + r] : __int_as_float(0x7f800000);
                    lim_s[8 * n + g] = p.causal ? r % p.L + S - p.L : S - 1;
                }
            }
            __syncthreads();
            for (int n = 0; n < nt; ++n) {
                const float2 qs = *reinterpret_cast<const float2*>(qs_s + 8 * n + 2 * t);
                const float2 nl = *reinterpret_cast<const float2*>(lse_s + 8 * n + 2 * t);
                const int2 lim = *reinterpret_cast<const int2*>(lim_s + 8 * n + 2 * t);
                if (!__any_sync(0xffffffffu, max(lim.x, lim.y) >= k0)) continue;
                float s[2][4] = {};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 x = qsm[0][n][i][lane];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        mma<Keys::kF16>(s[u], a[u][2 * i], x.x, x.y);
                        mma<Keys::kF16>(s[u], a[u][2 * i + 1], x.z, x.w);
                    }
                    if constexpr (F32) {
                        const uint4 y = qsm[PARTS - 1][n][i][lane];
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            mma<Keys::kF16>(s[u], a[u][2 * i], y.x, y.y);
                            mma<Keys::kF16>(s[u], a[u][2 * i + 1], y.z, y.w);
                        }
                    }
                }
                if (__any_sync(0xffffffffu, k0 + 31 > min(lim.x, lim.y))) {
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (k0 + 16 * u + g + 8 * (e >> 1) > (e & 1 ? lim.y : lim.x)) s[u][e] = neg_inf();
                }
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        acc[u][h] += fast_exp2(fmaf(s[u][2 * h], qs.x, -nl.x)) + fast_exp2(fmaf(s[u][2 * h + 1], qs.y, -nl.y));
            }
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            acc[u][h] += __shfl_xor_sync(0xffffffffu, acc[u][h], 1);
            acc[u][h] += __shfl_xor_sync(0xffffffffu, acc[u][h], 2);
        }
    // lane t of the quad writes half t >> 1, key g + 8 (t & 1)
    const float mine = t & 2 ? (t & 1 ? acc[1][1] : acc[1][0]) : (t & 1 ? acc[0][1] : acc[0][0]);
    const long long k = cta0 + 32 * warp + 16 * (t >> 1) + g + 8 * (t & 1);
    if (k < p.w_S) {
        const long long at = static_cast<long long>(bk) * p.w_S + k;
        const float old = p.w_in && k < S ? p.w_in[at] : 0.f;
        p.w_out[at] = k < S ? old + mine : 0.f;
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
struct WalkPlan {
    int R, nt, nrc, nkc, C;  // nt: n-tiles of 8 rows of walk_kernel, 0: block_kernel
    bool whole;              // walk_kernel: a CTA per segment
    bool scores;             // key weights from stored scores
    long long items;         // CTAs
    size_t prefix_off, ml_off, o_off, lse_off, score_off, total;
};

constexpr int kBlockRows = 32;   // rows per kv head from which block_kernel takes a call
constexpr int kScoreRows = 8;    // rows per kv head up to which scores are stored
constexpr int kWholeKeys = 512;  // table capacity up to which a CTA takes a whole segment
constexpr int kMinPer = 2;       // least units of a share

// walk_kernel: 8 rows per CTA, or 16 where a (sequence, kv head) has more than
// 8 (not for fp32 queries, whose fragments take twice the registers); as many
// CTAs as are resident together (4 per SM, 2 with 16 rows or fp32), each an equal
// share of all keys, or, over short tables, one per segment and no merge.
// block_kernel: 64 rows, key chunks for about four CTAs per SM, of at least 256 keys.
WalkPlan plan(const pa_shape& sh, bool q4, bool weights, int sm_count) {
    WalkPlan w;
    w.R = sh.H_q / sh.H_kv * sh.L;
    const bool f32 = sh.dtype == PA_F32;
    w.nt = w.R >= kBlockRows ? 0 : w.R > 8 && !f32 ? 2 : 1;
    const int rows_cta = w.nt ? 8 * w.nt : 16 * kWarps;
    w.nrc = (w.R + rows_cta - 1) / rows_cta;
    w.scores = weights && w.R <= kScoreRows;
    const long long cap = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    const long long segs = static_cast<long long>(sh.B) * sh.H_kv * w.nrc;
    const size_t rows = static_cast<size_t>(sh.B) * sh.H_kv * w.R;
    w.whole = w.nt && cap <= kWholeKeys;
    w.nkc = 1;
    w.C = 0;
    size_t slots = 0;  // rows of partial states
    if (w.nt) {
        int resident = resident_ctas(w.nt, q4, f32);
        if (!q4 && w.nt == 1 && w.R > 4) resident = 2;  // (shared memory: 16 KB stages per warp)
        w.items = w.whole ? segs : static_cast<long long>(sm_count) * resident;
        if (!w.whole) slots = static_cast<size_t>(w.items) * 2 * rows_cta;
    } else {
        long long nkc = (4ll * sm_count + segs - 1) / segs;
        const long long most = (cap + 255) / 256;
        nkc = nkc < most ? nkc : most;
        long long C = (cap + nkc - 1) / nkc;
        C = (C + kTK - 1) / kTK * kTK;
        w.C = static_cast<int>(C);
        w.nkc = static_cast<int>((cap + C - 1) / C);
        w.items = segs * w.nkc;
        if (w.nkc > 1) slots = rows * w.nkc;
    }
    size_t off = kFlagBytes;
    w.prefix_off = off;
    if (w.nt && !w.whole) off = align_up(off + (static_cast<size_t>(sh.B) + 2) * 4, 256);
    w.ml_off = off;
    off = align_up(off + slots * 16, 256);
    w.o_off = off;
    off = align_up(off + slots * kD * 4, 256);
    w.lse_off = off;
    if (weights) off = align_up(off + rows * 4, 256);
    w.score_off = off;
    if (w.scores) off = align_up(off + rows * cap * 4, 256);
    w.total = off;
    return w;
}

// Launches `kernel`, whose start may overlap the end of the kernel before it.
template <class... P, class... A>
bool launch_dependent(void (*kernel)(P...), long long grid, int threads, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

// The attention, its merge over key chunks, then the key weights.
template <class Keys, class Values, int NT, bool F32, bool A16, bool W>
pa_status launch_walk(const WalkParams& p, long long items, int device, cudaStream_t stream) {
    const size_t smem = walk_smem(Keys::kF16, p.R < 8 * NT ? p.R : 8 * NT);
    static int attr_done[64] = {0};
    if (!attr_done[device]) {
        if (cudaFuncSetAttribute(walk_kernel<Keys, Values, NT, F32, A16, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 walk_smem(Keys::kF16, 8 * NT)) != cudaSuccess)
            return PA_ERR_CUDA;
        attr_done[device] = 1;
    }
    walk_kernel<Keys, Values, NT, F32, A16, W><<<static_cast<unsigned>(items), kWarps * 32, smem, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <class Keys, class Values, int NT, bool F32>
pa_status launch_walk_for(const WalkParams& p, long long items, int device, cudaStream_t stream) {
    const bool a16 = p.ps % 16 == 0;
    if constexpr (NT == 1) {
        if (p.score) return a16 ? launch_walk<Keys, Values, NT, F32, true, true>(p, items, device, stream)
                                : launch_walk<Keys, Values, NT, F32, false, true>(p, items, device, stream);
    }
    return a16 ? launch_walk<Keys, Values, NT, F32, true, false>(p, items, device, stream)
               : launch_walk<Keys, Values, NT, F32, false, false>(p, items, device, stream);
}

template <bool Q4, bool F32>
pa_status launch_block(const WalkParams& p, long long items, int device, cudaStream_t stream) {
    static int attr_done[64] = {0};
    if (!attr_done[device]) {
        if (cudaFuncSetAttribute(block_kernel<Q4, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 4 * kTileBytes) != cudaSuccess)
            return PA_ERR_CUDA;
        attr_done[device] = 1;
    }
    block_kernel<Q4, F32><<<static_cast<unsigned>(items), kWarps * 32, 4 * kTileBytes, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// The key weights from the rows' log-sum-exp.
pa_status launch_weights(const WalkParams& p, bool q4, bool f32, cudaStream_t stream) {
    const long long bk = static_cast<long long>(p.B) * p.H_kv, ntile = (p.w_S + 32 * kWarps - 1) / (32 * kWarps);
    if (ntile * bk > INT_MAX) return PA_ERR_UNSUPPORTED;
    const unsigned grid = static_cast<unsigned>(ntile * bk);
    if (!q4)
        walk_weights_kernel<BfKeys, false><<<grid, kWarps * 32, 0, stream>>>(p, static_cast<int>(ntile));
    else if (f32)
        walk_weights_kernel<Q4Keys, true><<<grid, kWarps * 32, 0, stream>>>(p, static_cast<int>(ntile));
    else
        walk_weights_kernel<Q4Keys, false><<<grid, kWarps * 32, 0, stream>>>(p, static_cast<int>(ntile));
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status launch(const WalkParams& p, const WalkPlan& w, bool q4, bool f32, int device, cudaStream_t stream) {
    const long long bk = static_cast<long long>(p.B) * p.H_kv;
    const long long items = w.items, rows = bk * p.R;
    const long long per = w.scores ? 256 : 32 * kWarps, ntile = (p.w_S + per - 1) / per;
    if (items > INT_MAX || rows > INT_MAX || ntile * bk > INT_MAX) return PA_ERR_UNSUPPORTED;
    // the shares count units in an int
    if (w.nt && !w.whole && bk * p.nrc * (p.max_S / kUnit + 1) > INT_MAX / 2) return PA_ERR_UNSUPPORTED;
    pa_status st;
    if (w.nt == 0)
        st = !q4 ? launch_block<false, false>(p, items, device, stream)
                 : f32 ? launch_block<true, true>(p, items, device, stream)
                       : launch_block<true, false>(p, items, device, stream);
    else if (!q4)
        st = w.nt == 2 ? launch_walk_for<BfKeys, BfValues, 2, false>(p, items, device, stream)
                       : launch_walk_for<BfKeys, BfValues, 1, false>(p, items, device, stream);
    else if (f32)
        st = launch_walk_for<Q4Keys, Q4Values, 1, true>(p, items, device, stream);
    else
        st = w.nt == 2 ? launch_walk_for<Q4Keys, Q4Values, 2, false>(p, items, device, stream)
                       : launch_walk_for<Q4Keys, Q4Values, 1, false>(p, items, device, stream);
    if (st != PA_OK) return st;
    if (p.nkc > 1 && !launch_dependent(f32 ? block_combine_kernel<true> : block_combine_kernel<false>, (rows + 3) / 4, 128, stream, p))
        return PA_ERR_CUDA;
    if (w.nt && !w.whole) {
        const int rows_cta = 8 * w.nt;
        const long long grid = bk * p.nrc * (rows_cta < p.R ? rows_cta : p.R);
        if (!launch_dependent(f32 ? walk_combine_kernel<true> : walk_combine_kernel<false>, grid, kWarps * 32, stream, p, rows_cta))
            return PA_ERR_CUDA;
    }
    if (!p.w_out) return PA_OK;
    if (w.scores) return launch_dependent(walk_sum_kernel, ntile * bk, 256, stream, p, static_cast<int>(ntile)) ? PA_OK : PA_ERR_CUDA;
    return launch_weights(p, q4, f32, stream);
}

// Rows per kv head from which bf16 queries over 4-bit pages go to the tensor-core
// tiles of q4_tiles.cu.
constexpr int kTileRows = 48;

bool tiles_take(const pa_shape& sh, bool q4, int sm_count) {
    return q4 && sh.dtype == PA_BF16 && static_cast<long long>(sh.H_q / sh.H_kv) * sh.L >= kTileRows &&
           q4_tiles_supported(sh, sm_count);
}

// ---- whole prompts over 4-bit pages: bf16 copies and the bf16 tile kernel -------
// (exact: a 4-bit value is a bf16 number).  Where a kv head has half as many rows as
// keys or more, the copies cost less than what q4_tiles.cu spends per segment
// (G = 4, H_kv = 8, us, tiles against copies: 4 x 2048 rows over 600 keys 46, 38; 4 x
// 8192 over 2048 198, 145; 8 x 2080 over 1000 .. 8000 352, 382; 8 x 1040 209, 247; 1 x
// 8192 over 16000 436, 444).  Sequences go in groups whose copies fit kDenseBytes.
constexpr size_t kDenseBytes = size_t(1) << 30;

struct DensePlan {
    pa_shape sh;  // one group, over the dense copies
    size_t id_off, k_off, v_off, total;  // id: block table, then lengths
};

bool dense_take(const pa_shape& sh, bool q4, bool weights, int sm_count, DensePlan* t) {
    if (!q4 || weights || sh.dtype != PA_BF16) return false;
    const long long cap = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    const long long R = static_cast<long long>(sh.H_q / sh.H_kv) * sh.L;
    if (R < kTileRows || 2 * R < cap) return false;
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

pa_status dense_launch(const WalkCall& c, const DensePlan& t) {
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
    DensePlan d;
    if (dense_take(sh, q4, weights, sm_count, &d)) return d.total;
    if (tiles_take(sh, q4, sm_count)) {
        const size_t n = align_up(q4_tiles_workspace_bytes(sh, sm_count), 256);
        return n + (weights ? static_cast<size_t>(sh.B) * sh.H_q * sh.L * 4 : 0);
    }
    return plan(sh, q4, weights, sm_count).total;
}

pa_status walk_launch(const WalkCall& c) {
    const pa_shape& sh = c.sh;
    const bool tiles = tiles_take(sh, c.ks != nullptr, c.dev.sm_count);
    const WalkPlan w = plan(sh, c.ks != nullptr, c.w_out != nullptr, c.dev.sm_count);
    if (c.ws_bytes < walk_workspace_bytes(sh, c.ks != nullptr, c.w_out != nullptr, c.dev.sm_count)) return PA_ERR_WORKSPACE;
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
    p.whole = w.whole ? 1 : 0;
    p.min_per = kMinPer;
    p.prefix = reinterpret_cast<int*>(ws + w.prefix_off);
    p.max_S = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    p.scale_log2 = c.scale * 1.4426950408889634f;
    p.score = w.scores ? reinterpret_cast<float*>(ws + w.score_off) : nullptr;
    p.cap = p.max_S;
    DensePlan d;
    if (dense_take(sh, c.ks != nullptr, c.w_out != nullptr, c.dev.sm_count, &d)) return dense_launch(c, d);
    if (tiles) {
        if (c.w_out)
            p.lse = reinterpret_cast<float*>(ws + align_up(q4_tiles_workspace_bytes(sh, c.dev.sm_count), 256));
        const pa_status st = q4_tiles_launch(c, p.lse);
        return st != PA_OK || !c.w_out ? st : launch_weights(p, true, false, c.stream);
    }
    return launch(p, w, c.ks != nullptr, sh.dtype == PA_F32, c.dev.device, c.stream);
}

}  // namespace pa
