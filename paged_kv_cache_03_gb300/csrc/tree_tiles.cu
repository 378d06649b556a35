// tree_tiles.cu -- attention of drafted trees on tcgen05 tensor cores: bf16 queries over
// bf16 and 4-bit pages, fp32 queries over fp32 and 4-bit pages.
//
// The rows of a (sequence, kv head), r = (query head of the group, draft l), are R = G L
// consecutive rows of the query, cut into tiles of 128.  All of them see every position
// before the drafts, so a key tile needs no mask unless it holds drafts or lies at the end
// ("tail"); there a row's bits come out of its words of the tree's mask.
//   S = Q K^T,  P = 2^(scale S - m),  O += P V,  with a maximum m and the sum l per row;
//   O / l at the end.
// m is the largest score when it was last too low by 2^kSlack (or there was none): a weight
// does not wait for the scores behind it, and O is rescaled only then.
// bf16 pages: P rounded to bf16 (2^-8).  4-bit pages: K and V dequantised to f16 on chip
// (exact), Q scaled by a power of two into f16's range (exact), P rounded to f16 (2^-11, and
// 2^-32 of the row's largest).
// fp32: Q, K, V and P in two f16 parts each, x = h + l up to 2^-22 x, and products h h + h l
// + l h (l l is below 2^-22); every row is scaled into f16's range by a power of two, and K's
// scale is undone in the scores, V's in the weights.
//
// Layout on GB300: one CTA per SM.
//   * A segment is one query tile of one (sequence, kv head) over all its key tiles, or, over
//     bf16 pages by TMA, C query tiles on C neighbouring CTAs, which walk the same key tiles
//     at about the same time: K and V cross from HBM about once and the others of the C find
//     them in L2.  Nothing waits for a neighbour.
//   * The key tiles of all segments are cut into equal shares, one per CTA (C CTAs), so
//     ragged contexts leave no SM idle; a segment that crosses shares leaves fp32 partial
//     states that tree_merge_kernel joins.
//   * Two slots t = 0, 1, one softmax warpgroup each with one row per thread, have their own
//     P (over S), m and l, which are joined at the piece's end.  bf16 queries: each takes half
//     of every tile's keys into an O of its own, and S has two places.  fp32 queries: the tiles
//     go to the slots in turn, and there is one O.  Tensor cores cut what they add to towards
//     0, so products of all of a CTA's keys in one sum came 7e-6 short over 4000 fp32 keys and
//     8e-5 over 64000; a tile's products are a sum of their own, which its slot's warps add to
//     O, in fp32 rounding: 0.9e-6 at any length (256 rows 182 us, 172 in one sum; over 4 bits
//     49 and 51).  One warp issues Q K^T and one P V, so products run beside both softmaxes.
//   * The producer warps bring K and V into rings in the 128-byte swizzle that the MMA reads:
//     one lane per page box by TMA (bf16, pages of a multiple of 8 slots), 16-byte
//     asynchronous copies (other page sizes), or rows converted on the way (4 bits, fp32).
//   * One warp publishes the pieces of segments in a ring, with the bits of the slots that
//     hold drafts, and another loads the query tiles by TMA.
//   * Value rows that nobody sees (behind the context, slots without a draft) may hold
//     NaN, and 0 * NaN is NaN: copies leave zeros there, and behind TMA warp 1 zeroes them
//     before the tile is announced.
//   * All waits are bounded; on a timeout the CTA records PA_FLAG_TIMEOUT, frees its TMEM
//     and exits.
//
// Measured (G = 4, H_kv = 8, a call among others, with the merge):
//   64 sequences of 128 .. 4096 keys, 64 rows    89 us for 506 MB, 5.7 TB/s: HBM is 70% busy
//   16 of 32768, 128 rows, pages of 16          320 us, 6.7 TB/s: bound by HBM
//   16 of 1000 .. 8000, 252 rows                 76 us for 69 GFLOP, 900 TFLOP/s: a tile takes
//     1750 cycles, of them 1024 products at the peak rate; Q, K, V and TMA's stores pass
//     through shared memory in 1280.  Without exponentials it is no faster, without maxima
//     and sums 9%
//   32 of 500 .. 8000 in 4 bits, 96 rows         81 us: a tile takes 2170 cycles, the softmax
//     beside eight converting warps
//   8 of 1000 .. 8000 in fp32, 64 / 256 rows     94 / 182 us: conversion, 4500 cycles a tile of
//     64 keys, and three products, 3200
//   8 of 1000 .. 8000 in 4 bits, fp32, 64 rows   49 us: changes of segment, and 3500 cycles a
//     tile, of them 2048 products
#include <algorithm>
#include <cfloat>
#include <climits>
#include <mutex>

#include <cudaTypedefs.h>

#include "stage.cuh"
#include "tc.cuh"
#include "tree.h"

namespace pa {
namespace {

constexpr int kD = kHeadDim;
constexpr int BM = 128;  // query rows of a tile
// S of slot t at 128 t, O at 256 + 128 t; fp32 queries: O at 256, a tile's products at 384.
constexpr uint32_t kTmemCols = 512;
// What a segment's query load, first softmax and epilogue cost, in key tiles: the
// shares count it, or CTAs with many short segments would finish last.  (Of 64 sequences,
// 256 rows take 158, 154 and 151 us with 3, 4 and 5, 64 rows 91, 91 and 94.)
constexpr int kSegCost = 4;
// Least cost of a share.  Two tiles: one sequence of 2000 keys, 4 kv heads, 13 us of bf16 and
// 19 of fp32, with 8 of them 20 and 29.
constexpr int kMinPer = 2;
// Where there is a CTA for each segment and tables hold at most so many key tiles, segments
// stay whole and there is no merge: 4, or 8 where segments are for at least a quarter of the
// CTAs (whole and cut, bf16: 4 segments of 4 tiles 11.2 and 13, of 8 tiles 16.5 and 11.8; 120
// segments of 8 tiles 18 and 22; fp32: 32 of 8 tiles 31 and 25, 120 of them 28 and 35 us).
constexpr int kWholeFew = 4, kWholeMany = 8;
constexpr int kQTile = BM * kD * 2;
enum Bar {
    kQFull = 0,     // + buffer: the query tile is there (4 bit: as it is)
    kQEmpty = 2,    // + buffer: every Q K^T of its piece is done
    kKFull = 4,     // + slot
    kKEmpty = 7,    // + slot
    kVFull = 10,    // + slot
    kVEmpty = 13,   // + slot
    kVTail = 16,    // + slot: a tail tile's values are there, not yet cleaned (by TMA)
    kQReady = 16,   // + buffer: the query tile is there in f16 (f16 products; never with kVTail)
    kTFree = 18,    // a tile's products are in O (fp32 queries; never with kVTail)
    kSFull = 19,    // + place of S (halves) or slot
    kPFull = 21,    // + t + 2 x place
    kODone = 25,    // + t + 2 x place: O has taken in that P
    kOFree = 29,    // + t: the epilogue has read O
    kXFull = 31,    // both slots' maxima and sums are there
    kXFree = 32,    // ... and read
    kMmaDone = 33,
    kVScale = 34    // + tile & 3: the scales of V's rows are there (fp32 pages)
};
// bf16 queries: bf16 pages by TMA or by copies, 4-bit pages.  fp32 queries: fp32 pages,
// 4-bit pages.
enum Source { kTma, kCopy, kQ4, kF32, kQ4F };
constexpr bool fp32(Source s) { return s >= kF32; }
constexpr bool four_bit(Source s) { return s == kQ4 || s == kQ4F; }
constexpr bool is_f16(Source s) { return s >= kQ4; }  // the products' operands
// f16 parts of an operand: of Q (and P), of K and V.
constexpr int q_parts(Source s) { return fp32(s) ? 2 : 1; }
constexpr int kv_parts(Source s) { return s == kF32 ? 2 : 1; }
// Warps: K/V producers (rows that are converted: four for K, four for V), then four of MMA
// and pieces, then eight of softmax.
constexpr int producers(Source s) { return is_f16(s) ? 8 : 4; }
constexpr int threads(Source s) { return 32 * (producers(s) + 4 + 8); }
// K and V tiles in the rings.  Three: with C = 2 a tile's time is below the latency of HBM.
// 4-bit rows wait as they are, raw_stages tiles of them, and need the space for that.
constexpr int slots(Source s) { return is_f16(s) ? 2 : 3; }
// Keys of a tile: two parts of 128 would leave no room for a second tile.
constexpr int keys(Source s) { return s == kF32 ? 64 : 128; }
// bf16 queries: each slot takes half of every tile's keys, and S has two places, so a slot's
// softmax finds the next S there (with whole tiles in turn and one place each 256 rows of 64
// sequences took 154 us, not 139, and contexts of 100 .. 500 keys 43, not 34).  fp32 queries
// (products of three or two parts, which bound them): the slots take the tiles in turn.
constexpr bool halves(Source s) { return !fp32(s); }
constexpr int raw_stages(Source s) { return s == kQ4 ? 3 : s == kQ4F ? 1 : 0; }
// Published pieces: enough for producers that are that many tiles ahead, were each tile a
// piece.
constexpr int items(Source s) { return is_f16(s) ? 8 : 4; }
// The pieces' barriers: full + place, then empty + place.
constexpr int item_bars(Source s) { return s == kF32 ? kVScale + 4 : kVScale; }
// Registers of a thread by role: what setmaxnreg can share out, 512 x 128 or 640 x 96.
struct Regs {
    int producer, misc, softmax;
};
constexpr Regs regs(Source s) {
    return !is_f16(s) ? Regs{72, 104, 168} : s == kF32 ? Regs{104, 48, 112} : Regs{64, 64, 144};
}

constexpr int launch_regs(Source s) { return is_f16(s) ? 96 : 128; }  // what __launch_bounds__ leaves a thread
constexpr bool regs_fit(Source s) {
    const Regs r = regs(s);
    return 32 * (producers(s) * r.producer + 4 * r.misc + 8 * r.softmax) <= threads(s) * launch_regs(s);
}
static_assert(regs_fit(kTma) && regs_fit(kCopy) && regs_fit(kQ4) && regs_fit(kF32) && regs_fit(kQ4F),
              "an increase beyond what the others gave up would wait forever");

// Shared memory from a 1024-byte boundary (the attribute of smem_raw) on.  Q: one tile, or
// two of at most 64 rows that the pieces take in turn.
struct Smem {
    int k, v, raw, bar, items, tmem, abort, x, q_scale, o_max, kv_scale, total;
};
constexpr int kItemBytes = 168;
constexpr Smem smem(Source s) {
    Smem m{};
    int at = q_parts(s) * kQTile;
    m.k = at;  // [slot][part]
    at += slots(s) * kv_parts(s) * keys(s) * kD * 2;
    m.v = at;
    at += slots(s) * kv_parts(s) * keys(s) * kD * 2;
    m.raw = at;  // [producer warp][stage]
    at += 8 * raw_stages(s) * kRawStage;
    m.bar = at;
    at += (item_bars(s) + 2 * items(s)) * 8;
    m.items = at;
    at += items(s) * kItemBytes;
    m.tmem = at;
    m.abort = at + 8;
    at += 16;
    m.x = at;  // [2][128] maximum and sum; before that the share and the scan's sums
    at += 2 * BM * 8;
    m.q_scale = at;  // f16: [2][128] the inverse of a row's scale
    if (is_f16(s)) at += 2 * BM * 4;
    m.o_max = at;  // fp32 queries: [2 pieces][128] the maximum that O is relative to
    if (fp32(s)) at += 2 * BM * 4;
    // fp32 pages, a number per key: [8 tiles] K's inverse scale, [4 tiles] the exponent of V's
    // scale, [4 tiles] that scale
    m.kv_scale = at;
    if (s == kF32) at += (8 + 4 + 4) * keys(s) * 4;
    m.total = at;
    return m;
}
static_assert(smem(kTma).total <= 232448 && smem(kQ4).total <= 232448 && smem(kF32).total <= 232448 &&
                  smem(kQ4F).total <= 232448,
              "227 KB");
static_assert(smem(kQ4).raw % 16 == 0 && smem(kQ4F).raw % 16 == 0 && smem(kTma).x % 8 == 0 && smem(kF32).kv_scale % 16 == 0,
              "alignment");

struct TileParams {
    const uint8_t *kc, *ks, *vc, *vs;  // codes or rows, scales
    const float* q;                    // fp32 queries
    const int32_t* bt;
    const int32_t* ctx;
    const uint32_t* mask;
    void* out;
    uint32_t* flag;
    float2* part_ml;  // [2 per CTA][128]: max, sum
    float* part_o;    // [2 per CTA][128][D]
    int4* split;      // per share: the segment that starts in it and ends in a later one,
    int* join;        // and the share in which the segment that comes into it starts (-1: none)
    int B, H_kv, R, L, W, nG, num_pages, ps, max_npg;  // nG: groups of C query tiles
    int pool_rows, box;          // rows of the pool, of a K/V box
    int q_box, q_half, q_bufs;   // rows of a query box, bytes of 64 dims of a buffer, buffers
    long long max_S;
    float scale_log2;
    int out32;  // the output is 32-byte aligned
    int whole;  // a CTA (C CTAs) per segment
};

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// Length of a sequence, 0 for one that breaks the contract.
__device__ __forceinline__ int seq_len(const TileParams& p, int b) {
    const int S = __ldg(p.ctx + b);
    return S < p.L || static_cast<long long>(S) > p.max_S ? 0 : S;
}
template <int BN>
__device__ __forceinline__ int key_tiles(int S) {
    return (S + BN - 1) / BN;
}
template <int BN>
__device__ __forceinline__ int seq_cost(const TileParams& p, int S) {
    return S == 0 ? 0 : p.H_kv * p.nG * (kSegCost + key_tiles<BN>(S));
}

// A published piece: key tiles j0 .. j0 + n - 1 of its ng.  Place k % items holds piece k
// from kItemFull to kItemEmpty.
struct Item {
    int b, S, kvh, mp, ng, j0, n;  // n = 0: no more
    int before[2];      // the even and the odd tiles of earlier pieces (in turn: of slot t)
    uint32_t live[32];  // slots that hold a draft (pieces with tail tiles)
};
static_assert(sizeof(Item) <= kItemBytes && kItemBytes % 8 == 0, "item slot");

// A place in a ring of N and how often it has come round.
template <int N>
struct Ring {
    int s = 0;
    uint32_t phase = 0u;
    __device__ __forceinline__ void next() {
        if (++s == N) {
            s = 0;
            phase ^= 1u;
        }
    }
};

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}
__device__ __forceinline__ bool aborted(volatile int* f) { return __any_sync(0xffffffffu, *f != 0); }
__device__ __forceinline__ void give_up(const TileParams& p, volatile int* f) {
    *f = 1;
    atomicOr(p.flag, PA_FLAG_TIMEOUT);
}

constexpr uint32_t idesc(bool f16, int n, int b_mn) {
    return tc::idesc_bf16(BM, n, 0, b_mn) & ~(f16 ? (1u << 7) | (1u << 10) : 0u);
}

__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
// A pair of numbers in f16's range in two f16 parts.
__device__ __forceinline__ void split_f16(float2 x, uint32_t& hi, uint32_t& lo) {
    const float2 h = make_float2(__uint_as_float(__float_as_uint(x.x) & 0xffffe000u),
                                 __uint_as_float(__float_as_uint(x.y) & 0xffffe000u));
    hi = pack_f16x2(h.x, h.y);
    lo = pack_f16x2(x.x - h.x, x.y - h.y);
}
// k of 2^k (a normal number).
__device__ __forceinline__ float exponent_of(float x) { return static_cast<float>(static_cast<int>(__float_as_uint(x) >> 23) - 127); }

// A warp's registers from here on (a warpgroup together): fewer than at the launch, or more.
template <int N, int LAUNCH>
__device__ __forceinline__ void reg_set() {
    static_assert(N % 8 == 0 && N >= 24 && N <= 256, "setmaxnreg");
    if constexpr (N <= LAUNCH) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

template <Source SRC, int C>
__global__ void __launch_bounds__(threads(SRC), 1)
    tree_tile_kernel(const TileParams p, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
    constexpr bool F16 = is_f16(SRC), F32 = fp32(SRC);
    constexpr int kThreads = threads(SRC), kProd = producers(SRC), N = slots(SRC), I = items(SRC);
    constexpr int BN = keys(SRC), kTile = BN * kD * 2;
    constexpr bool HALF = halves(SRC);
    constexpr int UK = HALF ? BN / 2 : BN;  // keys of a slot's P
    constexpr int QP = q_parts(SRC), VP = kv_parts(SRC), kRing = VP * kTile;
    constexpr int kItemFull = item_bars(SRC), kItemEmpty = kItemFull + I;
    constexpr Smem M = smem(SRC);
    // Tiles behind TMA: [8 rows][64-dim half][row][128 bytes], as boxes of rows come; else
    // [half][BN rows][128 bytes].
    constexpr uint32_t kHalf = SRC == kTma ? 1024u : BN * 128u, kGroup = SRC == kTma ? 2048u : 1024u;
    // By TMA, K and V of C > 1 tiles come from a warp each, so that K is read ahead of V (256
    // rows: 142 us from one warp, 136 from two), else from one (at the rate of HBM: 320 and 327).
    constexpr bool kApart = C > 1;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = smem_u32(smem_raw);
    auto bar = [&](int i) { return base + M.bar + 8u * static_cast<uint32_t>(i); };
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem_raw + M.abort);
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + M.tmem);
    // all units, units per share, first sequence, its first unit; [4 ..): sums of a scan
    int* const share = reinterpret_cast<int*>(smem_raw + M.x);
    int* const sums = share + 4;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(blockIdx.x) % C;  // which of the C query tiles
    const int my_share = static_cast<int>(blockIdx.x) / C, shares = static_cast<int>(gridDim.x) / C;
    pdl_launch_dependents();

    // ---- set-up ----------------------------------------------------------------
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(kQFull + s), 1);
            if (F16) mbar_init(bar(kQReady + s), 4);
            mbar_init(bar(kQEmpty + s), 1);
            mbar_init(bar(kSFull + s), 1);
            for (int b = 0; b < 4; b += 2) {
                mbar_init(bar(kPFull + s + b), 4);
                mbar_init(bar(kODone + s + b), 1);
            }
            mbar_init(bar(kOFree + s), 8);
            mbar_init(bar(kXFull + s), 8);  // (and kXFree)
        }
        if (F32) mbar_init(bar(kTFree), 4);
        for (int s = 0; s < N; ++s) {
            mbar_init(bar(kKFull + s), SRC == kTma ? 1 : 4);
            mbar_init(bar(kKEmpty + s), 1);
            mbar_init(bar(kVFull + s), SRC == kTma ? 1 : 4);
            mbar_init(bar(kVEmpty + s), 1);
            if (SRC == kTma) mbar_init(bar(kVTail + s), 1);
        }
        if (SRC == kF32)
            for (int s = 0; s < 4; ++s) mbar_init(bar(kVScale + s), 4);
        mbar_init(bar(kMmaDone), 2);
        for (int s = 0; s < I; ++s) {
            mbar_init(bar(kItemFull + s), 1);
            // K/V warps, the MMA warps, the query warp, softmax warps
            mbar_init(bar(kItemEmpty + s), (SRC != kTma ? kProd : kApart ? 3 : 2) + 3 + 8);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kProd) {
        tc::tmem_alloc(base + M.tmem, kTmemCols);
        tc::tmem_relinquish();
    }
    // ---- this share ----------------------------------------------------------------
    if (p.whole) {
        // segment i: a share that holds it and no other
        if (tid == 0) {
            const int b = my_share / (p.H_kv * p.nG), cost = kSegCost + key_tiles<BN>(seq_len(p, b));
            share[0] = INT_MAX;
            share[1] = cost;
            share[2] = b;
        }
    } else {
        int mine = 0, v = 0;
        for (int b = tid; b < p.B; b += kThreads) {
            const int n = seq_cost<BN>(p, seq_len(p, b));
            if (b == tid) mine = n;
            v += n;
        }
        v = __reduce_add_sync(0xffffffffu, v);
        if (lane == 0) sums[warp] = v;
        __syncthreads();
        int total = 0;
        for (int w = 0; w < kThreads / 32; ++w) total += sums[w];
        const int per = max((total + shares - 1) / shares, kMinPer);
        const int u = my_share * per;
        if (tid == 0) {
            share[0] = total;
            share[1] = per;
        }
        int carry = 0;
        for (int b0 = 0; b0 < p.B; b0 += kThreads) {
            const int b = b0 + tid;
            int x = mine;
            if (b0 > 0) x = b < p.B ? seq_cost<BN>(p, seq_len(p, b)) : 0;
            int incl = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            __syncthreads();
            if (lane == 31) sums[warp] = incl;
            __syncthreads();
            int before = carry + incl - x;
            for (int w = 0; w < warp; ++w) before += sums[w];
            if (b < p.B && before <= u && u < before + x) {
                share[2] = b;
                share[3] = before;
            }
            for (int w = 0; w < kThreads / 32; ++w) carry += sums[w];
        }
    }
    {
        // sequences that break the contract: zero rows
        for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
            if (seq_len(p, b) > 0) continue;
            if (tid == 0) atomicOr(p.flag, PA_FLAG_BAD_CONTEXT);
            const long long rows = static_cast<long long>(p.H_kv) * p.R;
            constexpr int kVecs = F32 ? kD / 4 : kD / 8;  // 16 bytes each
            uint4* const o = static_cast<uint4*>(p.out) + b * rows * kVecs;
            for (long long i = tid; i < rows * kVecs; i += kThreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const int total = share[0], per = share[1], first_b = share[2], first_unit = p.whole ? 0 : share[3];
    // which slots of the share's first sequence hold a draft, where one warp would take long
    uint32_t first_live = 0u;
    if (p.W > 4 && (p.whole || my_share * per < total)) {
        uint32_t* const words = reinterpret_cast<uint32_t*>(share) + 64;
        if (tid < 32) words[tid] = 0u;
        __syncthreads();
        const uint32_t* const mask = p.mask + static_cast<long long>(first_b) * p.L * p.W;
#pragma unroll 4
        for (int i = warp; i < p.L; i += kThreads / 32) {
            const uint32_t word = lane < p.W ? __ldg(mask + static_cast<long long>(i) * p.W + lane) : 0u;
            if (__any_sync(0xffffffffu, word != 0u) && lane == 0) atomicOr(words + (i >> 5), 1u << (i & 31));
        }
        __syncthreads();
        first_live = words[lane];
    }
    __syncthreads();  // (the states lie there)
    auto slot = [&](int k) { return reinterpret_cast<volatile Item*>(smem_raw + M.items + kItemBytes * (k % I)); };
    auto take = [&](int k) { return warp_wait(bar(kItemFull + k % I), (k / I) & 1); };  // a whole warp
    auto release = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kItemEmpty + k % I));
    };
    // key tiles of a piece from this one on hold drafts or the context's end
    auto first_tail = [&](int S) { return (S - p.L) / BN; };
    // query buffer of a piece, and how often it has come round
    auto q_buf = [&](int k) { return p.q_bufs == 2 ? k & 1 : 0; };
    auto q_use = [&](int k) { return p.q_bufs == 2 ? k >> 1 : k; };

    if (warp < kProd) {
        // ========================= K/V producers ==================================
        reg_set<regs(SRC).producer, launch_regs(SRC)>();
        bool ok = true;
        if constexpr (SRC == kTma) {
            if (warp == 0 || (kApart && warp == 2)) {
                const bool keys = warp == 0, values = !kApart || warp == 2;
                // (read once, or by C CTAs close together: 256 rows of a head 136 us, kept to the last 141)
                const uint64_t policy = p.nG == 1 ? l2_policy_evict_first() : l2_policy_evict_last();
                const int nbox = BN / p.box;
                bool bad_page = false;
                Ring<N> g;
                for (int k = 0; ok; ++k) {
                    ok = take(k);
                    if (!ok) break;
                    const int n = slot(k)->n, j0 = slot(k)->j0, b = slot(k)->b, S = slot(k)->S, kvh = slot(k)->kvh;
                    release(k);
                    if (n == 0) break;
                    const int32_t* const table = p.bt + static_cast<long long>(b) * p.max_npg;
                    const int tail = first_tail(S);
                    // lane i brings box i of a tile; its page id is requested a tile ahead
                    auto page_of = [&](int j) {
                        const int key = j * BN + lane * p.box;
                        return lane < nbox && key < S ? __ldg(table + key / p.ps) : 0;
                    };
                    int page = page_of(j0);
                    for (int j = j0; j < j0 + n; ++j, g.next()) {
                        const int key = j * BN + lane * p.box;
                        const bool there = lane < nbox && key < S;
                        const bool good = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages);
                        bad_page |= there && !good;
                        // (groups of 8 rows; those behind the pool read as zeros)
                        const int row = (good ? (page * p.H_kv + kvh) * p.ps + key % p.ps : p.pool_rows) >> 3;
                        const uint32_t bytes = static_cast<uint32_t>(min(nbox, (S - j * BN + p.box - 1) / p.box)) * p.box * 256u;
                        if (j + 1 < j0 + n) page = page_of(j + 1);
                        auto load = [&](int empty, int full, uint32_t ring, const CUtensorMap* map) {
                            if (!warp_wait(bar(empty + g.s), g.phase ^ 1u) || aborted(abort_flag)) return false;
                            if (lane == 0) mbar_arrive_expect_tx(bar(full + g.s), bytes);
                            __syncwarp();
                            if (there)
                                tc::tma_load_4d(base + ring + g.s * kTile + lane * p.box * 256, map, 0, 0, 0, row, bar(full + g.s),
                                                policy);
                            return true;
                        };
                        ok = (!keys || load(kKEmpty, kKFull, M.k, &kmap)) &&
                             (!values || load(kVEmpty, j >= tail ? kVTail : kVFull, M.v, &vmap));
                        if (!ok) break;
                    }
                }
                // Without an error every copy has been waited for by the MMA warps.  With one,
                // give those in flight time to land before the shared memory goes.
                if (!ok)
                    for (int s = 0; s < N; ++s) {
                        if (keys) mbar_wait_for(bar(kKFull + s), g.phase ^ (s >= g.s), 50000000ull);
                        if (values) mbar_wait_for(bar(kVFull + s), g.phase ^ (s >= g.s), 50000000ull);
                    }
                if (__any_sync(0xffffffffu, bad_page) && lane == 0) atomicOr(p.flag, PA_FLAG_BAD_PAGE);
            } else if (warp == 1) {
                // value rows of tail tiles that nobody sees
                Ring<N> g;
                uint32_t phases = 0u;  // of the slots' tail barriers
                for (int k = 0; ok; ++k) {
                    ok = take(k);
                    if (!ok) break;
                    const int n = slot(k)->n, j0 = slot(k)->j0, S = slot(k)->S, first = S - p.L, tail = first_tail(S);
                    for (int j = j0; j < j0 + n; ++j, g.next()) {
                        if (j < tail) continue;
                        ok = warp_wait(bar(kVTail + g.s), phases >> g.s & 1u);
                        if (!ok) break;
                        phases ^= 1u << g.s;
#pragma unroll 1
                        for (int r = lane; r < BN; r += 32) {
                            const int x = j * BN + r - first;  // draft
                            if (x < 0 || (x < p.L && (slot(k)->live[x >> 5] >> (x & 31) & 1u))) continue;
                            const uint32_t at = base + M.v + g.s * kTile + (r >> 3) * kGroup + (r & 7) * 128;
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                sts128(at + 16 * c, 0u, 0u, 0u, 0u);
                                sts128(at + kHalf + 16 * c, 0u, 0u, 0u, 0u);
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(kVFull + g.s));
                    }
                    release(k);
                    if (!ok || n == 0 || aborted(abort_flag)) break;
                }
            }
        } else {
            // pool rows of the next tile, lane 8 i + r: key 32 i + 8 (warp & 3) + r; -1 where
            // nobody sees the key
            int page = 0, in_page = -1, row_base = 0;
            bool bad_page = false;
            auto lookup = [&](int k, int j) {
                const volatile Item* const it = slot(k);
                const int key = j * BN + 32 * (lane >> 3) + 8 * (warp & 3) + (lane & 7), lp = key / p.ps;
                const int S = it->S, x = key - (S - p.L);
                const bool seen = key < S && (lane >> 3) < BN / 32 && (x < 0 || (it->live[x >> 5] >> (x & 31) & 1u));
                in_page = seen ? key - lp * p.ps : -1;
                page = seen ? __ldg(p.bt + static_cast<long long>(it->b) * p.max_npg + lp) : 0;
                row_base = it->kvh;
            };
            auto rows_of = [&]() {
                const bool good = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages);
                bad_page |= in_page >= 0 && !good;
                return in_page >= 0 && good ? (page * p.H_kv + row_base) * p.ps + in_page : -1;
            };
            auto announce = [&](int x) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(x));
            };
            int k = 0, j = 0, last = -1;
            ok = take(0);
            bool more = ok && slot(0)->n > 0;
            if (more) {
                j = slot(0)->j0;
                last = j + slot(0)->n - 1;
                lookup(0, j);
            }
            // the tile after tile j of piece k: its page ids are requested now
            auto next = [&]() {
                if (j < last) {
                    ++j;
                } else {
                    release(k);
                    ++k;
                    ok = take(k);
                    if (!ok) {
                        more = false;
                        return;
                    }
                    more = slot(k)->n > 0;
                    j = slot(k)->j0;
                    last = j + slot(k)->n - 1;
                }
                if (more) lookup(k, j);
            };
            Ring<N> g;
            if constexpr (four_bit(SRC)) {
                constexpr int kRawStages = raw_stages(SRC);
                // Warps 0-3 dequantise K, 4-7 V.  A tile's 4-bit rows are copied to the warp's
                // staging kRawStages tiles ahead.
                const bool is_v = warp >= 4;
                const uint32_t stages = base + M.raw + warp * kRawStages * kRawStage, ring = base + (is_v ? M.v : M.k);
                const uint8_t *const codes = is_v ? p.vc : p.kc, *const scales = is_v ? p.vs : p.ks;
                const int full = is_v ? kVFull : kKFull, empty = is_v ? kVEmpty : kKEmpty;
                RawTile t;
                Ring<kRawStages> r;
                int ahead = 0;  // tiles on their way
                auto request = [&](int stage) {  // ... the next one (an empty group past the last)
                    if (more) {
                        const int rows = rows_of();
                        RawTile::copy(stages + stage * kRawStage, codes, scales, rows, lane);
                        ++ahead;
                        next();
                    }
                    cp_async_commit();
                };
                for (int i = 0; i < kRawStages; ++i) request(i);
                while (ok && ahead > 0) {
                    cp_async_wait<kRawStages - 1>();
                    __syncwarp();
                    t.read(stages + r.s * kRawStage, lane);
                    --ahead;
                    ok = warp_wait(bar(empty + g.s), g.phase ^ 1u);
                    if (!ok || aborted(abort_flag)) break;
                    t.store<false>(ring + g.s * kTile, warp & 3, lane);
                    announce(full + g.s);
                    g.next();
                    // (after that: the piece it may have to wait for can need this tile)
                    request(r.s);
                    r.next();
                }
                cp_async_wait<0>();
            } else if constexpr (SRC == kF32) {
                // Warps 0-3 bring K, 4-7 V: warp w rows 32 i + 8 w .., i = 0, 1, which are loaded a
                // tile ahead.  A row is taken by a power of two so that its largest value lies in
                // [2^14, 2^15), and stored in two f16 parts: all but 2^-22 of a value, or 2^-40 of
                // the row's largest.  Scores are scaled back by key; V's scale goes into P, so it is
                // announced before V's place in the ring is free.
                const bool is_v = warp >= 4;
                const int w = warp & 3;
                const float* const pool = reinterpret_cast<const float*>(is_v ? p.vc : p.kc);
                const uint32_t ring = base + (is_v ? M.v : M.k);
                const int full = is_v ? kVFull : kKFull, empty = is_v ? kVEmpty : kKEmpty;
                float* const scales = reinterpret_cast<float*>(smem_raw + M.kv_scale) + (is_v ? 8 * BN : 0);
                // Row of 8 and dims 16 q + 4 l4 ..: 16 lanes take every other row, so that their 8-byte
                // stores hit all banks once.
                const int r8 = (lane >> 2 & 3) * 2 + (lane >> 4), l4 = lane & 3;
                auto prefetch = [&](int rows) {
                    if (rows >= 0) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) prefetch_l2(pool + static_cast<long long>(rows) * kD + 32 * i);
                    }
                };
                auto load = [&](float4 (&v)[8], int rows, int i) {
                    const int row = __shfl_sync(0xffffffffu, rows, 8 * i + r8);
                    const float4* const src = reinterpret_cast<const float4*>(pool + (row < 0 ? 0 : static_cast<long long>(row) * kD)) + l4;
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[q] = row < 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : __ldcs(src + 4 * q);
                };
                auto largest_of = [&](const float4 (&v)[8]) {  // of the row: its four lanes
                    float mx = 0.f;
#pragma unroll
                    for (int q = 0; q < 8; ++q) mx = fmax3(fmax3(mx, fabsf(v[q].x), fabsf(v[q].y)), fabsf(v[q].z), fabsf(v[q].w));
#pragma unroll
                    for (int d = 1; d < 4; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                    return mx;
                };
                auto store = [&](const float4 (&v)[8], int i, float up) {
                    const uint32_t at = ring + g.s * kRing + (32 * i + 8 * w + r8) * 128 + (l4 & 1) * 8;
                    const float2 up2 = make_float2(up, up);
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const float2 x[2] = {__fmul2_rn(make_float2(v[q].x, v[q].y), up2),
                                             __fmul2_rn(make_float2(v[q].z, v[q].w), up2)};
                        uint32_t hi[2], lo[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) split_f16(x[e], hi[e], lo[e]);
                        const int c = (4 * q + l4) >> 1;  // chunk of 8 dims
                        const uint32_t to = at + (c >> 3) * kHalf + (((c & 7) ^ r8) << 4);
                        sts64(to, hi[0], hi[1]);
                        sts64(to + kTile, lo[0], lo[1]);
                    }
                };
                float4 a[8], b[8];
                // of a row: the factor, kept for the softmax, of K inverted, of V with its exponent
                auto scale_of = [&](float mx, float* out) {
                    float up, down;
                    f16_scale(mx, up, down);
                    // At most 2^80, so that the sum of P 2^v (P below 2^16) stays a number; for zeros
                    // just that: they leave the maximum to keys that the output is made of.  (P is 0
                    // below 2^-126: a key whose values are 2^k times smaller than another's is lost to
                    // the sum where it weighs less than 2^(k - 133) of that one.)
                    if (is_v) up = mx == 0.f ? 1.2089258e24f : fminf(up, 1.2089258e24f);
                    if (l4 == 0) {
                        *out = is_v ? exponent_of(up) : down;
                        if (is_v) out[4 * BN] = up;
                    }
                    return up;
                };
                // rows of this tile; page ids of the next one are always on their way
                int tile = 0;
                bool there = more;
                if (more) {
                    const int rows = rows_of();
                    load(a, rows, 0);
                    load(b, rows, 1);
                    next();
                }
                while (ok && there) {
                    there = more;
                    const int rows = more ? rows_of() : -1;  // of the tile after
                    prefetch(rows);
                    if (more) next();
                    if (!ok) break;
                    // (K's may be written while the softmax of four tiles before is under way, V's
                    // of three)
                    float* const mine = scales + (tile & (is_v ? 3 : 7)) * BN + 8 * w + r8;
                    const float up0 = scale_of(largest_of(a), mine), up1 = scale_of(largest_of(b), mine + 32);
                    __syncwarp();
                    if (is_v && lane == 0) mbar_arrive(bar(kVScale + (tile & 3)));
                    ok = warp_wait(bar(empty + g.s), g.phase ^ 1u);
                    if (!ok || aborted(abort_flag)) break;
                    store(a, 0, up0);
                    load(a, rows, 0);
                    store(b, 1, up1);
                    load(b, rows, 1);
                    announce(full + g.s);
                    ++tile;
                    g.next();
                }
            } else {
                // K and V of a tile are one group of copies; a tile is announced when the next
                // one is requested.
                Ring<N> a;
                int pending = 0;
                auto finish = [&]() {
                    announce(kKFull + a.s);
                    announce(kVFull + a.s);
                    a.next();
                    --pending;
                };
                while (more) {
                    const int rows = rows_of();
                    next();
                    if (!ok) break;
                    ok = warp_wait(bar(kKEmpty + g.s), g.phase ^ 1u);
                    if (!ok || aborted(abort_flag)) break;
                    copy_tile(base + M.k + g.s * kTile, p.kc, rows, warp, lane);
                    ok = warp_wait(bar(kVEmpty + g.s), g.phase ^ 1u);
                    if (!ok || aborted(abort_flag)) break;
                    copy_tile(base + M.v + g.s * kTile, p.vc, rows, warp, lane);
                    cp_async_commit();
                    g.next();
                    if (++pending == N - 1) {
                        cp_async_wait<N - 2>();
                        finish();
                    }
                }
                cp_async_wait<0>();
                while (ok && pending > 0) finish();
            }
            if (__any_sync(0xffffffffu, bad_page) && lane == 0) atomicOr(p.flag, PA_FLAG_BAD_PAGE);
        }
        if (!ok && lane == 0) give_up(p, abort_flag);
    } else if (warp < kProd + 4) {
        reg_set<regs(SRC).misc, launch_regs(SRC)>();
        if (warp < kProd + 2) {
            // ========================== MMA issuers ==============================
            // One warp for Q K^T, one for P V: what one spends on waits and issues, the other
            // fills (one warp for both: 2000 cycles a tile of which the products are 1024).
            // The whole warp runs the loop and one elected lane issues.
            constexpr uint32_t idS = idesc(F16, BN, 0);  // Q, K both K-major
            constexpr uint32_t idO = idesc(F16, kD, 1);  // P K-major, V MN-major
            const uint64_t dQ0 = tc::smem_desc_sw128(base, 16, 1024);
            const uint64_t dK0 = tc::smem_desc_sw128(base + M.k, 16, kGroup);
            const uint64_t dV0 = tc::smem_desc_sw128(base + M.v, kHalf, kGroup);
            const bool leader = elect_one(), values = warp != kProd;
            Ring<N> ring;
            int g0 = 0, u0 = 0, u1 = 0, oe = 0;  // of earlier pieces: tiles, of each slot, epilogues
            bool ok = true;
            for (int k = 0; ok; ++k) {
                ok = take(k);
                if (!ok) break;
                const int n = slot(k)->n;
                release(k);
                if (n == 0) break;
                if (!values) {
                    const int buf = q_buf(k);
                    const uint64_t dq0 = tc::desc_advance(dQ0, buf * (QP * kQTile / 2)), dq1 = tc::desc_advance(dq0, p.q_half);
                    ok = warp_wait(bar((F16 ? kQReady : kQFull) + buf), q_use(k) & 1);
                    for (int i = 0; ok && i < n; ++i, ring.next()) {
                        // the place of S, and how often it was used
                        const int place = (HALF ? g0 + i : i) & 1, use = HALF ? (g0 + i) >> 1 : (i & 1 ? u1 : u0) + (i >> 1);
                        ok = warp_wait(bar(kKFull + ring.s), ring.phase);
                        // (its P V, and with halves that of the other slot before it, has read P)
                        if (ok && use > 0) ok = warp_wait(bar(kODone + (HALF ? 1 + 2 * place : place)), (use - 1) & 1);
                        if (!ok) break;
                        tc::fence_after_sync();
                        const uint64_t dk = tc::desc_advance(dK0, ring.s * kRing);
                        const uint32_t d = tmem + 128u * place;
                        if (leader) {
                            // the products of the parts, the smallest first (low x low is left out)
#pragma unroll
                            for (int part = QP + VP - 2; part >= 0; --part) {
                                const uint64_t qa = part == 1 ? tc::desc_advance(dq0, 2 * p.q_half) : dq0;
                                const uint64_t qb = part == 1 ? tc::desc_advance(dq1, 2 * p.q_half) : dq1;
                                const uint64_t ka = part == 2 ? tc::desc_advance(dk, kTile) : dk;
#pragma unroll
                                for (int kk = 0; kk < kD / 16; ++kk) {
                                    const uint64_t x = tc::desc_advance(kk < 4 ? qa : qb, (kk & 3) * 32);
                                    const uint64_t y = tc::desc_advance(ka, (kk >> 2) * kHalf + (kk & 3) * 32);
                                    if (kk == 0 && part == QP + VP - 2) tc::mma_bf16_c<0>(d, x, y, idS);
                                    else tc::mma_bf16_c<1>(d, x, y, idS);
                                }
                            }
                            tc::commit(bar(kSFull + place));
                            tc::commit(bar(kKEmpty + ring.s));
                            if (i == n - 1) tc::commit(bar(kQEmpty + buf));
                        }
                        __syncwarp();
                    }
                } else {
                    for (int i = 0; ok && i < n; ++i, ring.next()) {
                        ok = warp_wait(bar(kVFull + ring.s), ring.phase);
                        const uint64_t dv = tc::desc_advance(dV0, ring.s * kRing);
#pragma unroll
                        for (int h = 0; h < (HALF ? 2 : 1); ++h) {
                            const int t = HALF ? h : i & 1;  // the slot
                            const int b = HALF ? (g0 + i) & 1 : 0, use = HALF ? (g0 + i) >> 1 : (t ? u1 : u0) + (i >> 1);
                            ok = ok && warp_wait(bar(kPFull + t + 2 * b), use & 1);
                            // the previous piece's epilogue has read O
                            if (ok && i == 0 && oe > 0) ok = warp_wait(bar(kOFree + t), (oe - 1) & 1);
                            // the tile before has been added to O
                            if (!HALF && ok && i > 0) ok = warp_wait(bar(kTFree), (g0 + i - 1) & 1);
                            if (!ok) break;
                            tc::fence_after_sync();
                            const uint32_t d = tmem + 256u + 128u * (HALF ? t : i > 0), a = tmem + (HALF ? 128u * b + UK * t : 128u * t);
                            if (leader) {
#pragma unroll
                                for (int part = QP + VP - 2; part >= 0; --part) {
                                    // two parts of P: 16 columns of each for 32 keys
                                    const uint32_t pa = a + (part == 1 ? 16u : 0u);
                                    const uint64_t va = part == 2 ? tc::desc_advance(dv, kTile) : dv;
#pragma unroll
                                    for (int kk = 0; kk < UK / 16; ++kk) {
                                        const uint32_t x = pa + (QP == 1 ? kk * 8 : (kk >> 1) * 32 + (kk & 1) * 8);
                                        const uint64_t y = tc::desc_advance(va, (h * (UK / 16) + kk) * 2 * kGroup);
                                        if (kk == 0 && part == QP + VP - 2) tc::mma_bf16_ts(d, x, y, idO, HALF && i > 0);
                                        else tc::mma_bf16_ts_c<1>(d, x, y, idO);
                                    }
                                }
                                tc::commit(bar(kODone + t + 2 * b));
                                if (!HALF || h == 1) tc::commit(bar(kVEmpty + ring.s));
                            }
                            __syncwarp();
                        }
                        if (!ok) break;
                    }
                }
                if (!ok) break;
                g0 += n;
                u0 += (n + 1) >> 1;
                u1 += n >> 1;
                ++oe;
            }
            if (!ok && lane == 0) give_up(p, abort_flag);
            // nothing of ours may still be running when TMEM is freed
            if (leader) tc::commit(bar(kMmaDone));
            __syncwarp();
            if (!warp_wait(bar(kMmaDone), 0) && lane == 0) give_up(p, abort_flag);
        } else if (warp == kProd + 2) {
            // ========================= query tiles ===================================
            const uint64_t policy = l2_policy_evict_first();
            bool ok = true;
            int last = -1;  // piece whose query tile was asked for
            for (int k = 0;; ++k) {
                ok = take(k);
                if (!ok || slot(k)->n == 0) break;
                // when the products of the last piece in the buffer are done
                const int buf = q_buf(k), use = q_use(k), m = slot(k)->mp * C + rank;
                const int row = (slot(k)->b * p.H_kv + slot(k)->kvh) * p.R + m * BM;
                release(k);
                if constexpr (F32) continue;  // (the softmax warps load them)
                ok = use == 0 || warp_wait(bar(kQEmpty + buf), (use - 1) & 1);
                if (!ok || aborted(abort_flag)) break;
                if (lane == 0) {
                    if (m * BM < p.R) {
                        const uint32_t dst = base + buf * (kQTile / 2);
                        mbar_arrive_expect_tx(bar(kQFull + buf), static_cast<uint32_t>(p.q_box) * 256u);
                        tc::tma_load_2d(dst, &qmap, 0, row, bar(kQFull + buf), policy);
                        tc::tma_load_2d(dst + p.q_half, &qmap, 64, row, bar(kQFull + buf), policy);
                    } else {  // no rows for this CTA: its products are not looked at
                        mbar_arrive(bar(kQFull + buf));
                    }
                }
                last = k;
                __syncwarp();
            }
            // What an error elsewhere left in flight lands before the shared memory goes: the last
            // tile of each buffer.
            for (int k = max(0, last - p.q_bufs + 1); k <= last; ++k) mbar_wait_for(bar(kQFull + q_buf(k)), q_use(k) & 1, 50000000ull);
            if (!ok && lane == 0) give_up(p, abort_flag);
        } else if (warp == kProd + 3) {
            // ============================ pieces =====================================
            const int start = p.whole ? 0 : my_share * per, end = p.whole ? per : min(start + per, total);
            int b = 0, S = 0, kvh = 0, mp = 0, ng = 0, seg = end;  // seg: first position of the segment
            if (start < end) {
                b = first_b;
                S = seq_len(p, b);
                ng = key_tiles<BN>(S);
                const int i = p.whole ? my_share % (p.H_kv * p.nG) : (start - first_unit) / (kSegCost + ng);
                kvh = i / p.nG;
                mp = i - kvh * p.nG;
                seg = p.whole ? 0 : first_unit + i * (kSegCost + ng);
            }
            int4 crossing = make_int4(-1, 0, 0, 0);
            int from = -1;  // the share in which the segment that comes into this one starts
            int before0 = 0, before1 = 0;
            // lane w: word w of the slots of sequence live_b that hold a draft
            int live_b = start < end ? first_b : -1;
            uint32_t live = first_live;
            if (p.W <= 4) live_b = -1;
            bool ok = true;
            for (int k = 0;; ++k) {
                // this share's key tiles of the segment (none: the share ends before them)
                int j0 = 0, n = 0;
                if (seg < end) {
                    j0 = max(0, start - seg - kSegCost);
                    n = max(0, min(ng, end - seg - kSegCost) - j0);
                }
                if (k >= I && !warp_wait(bar(kItemEmpty + k % I), (k / I - 1) & 1)) {
                    ok = false;
                    break;
                }
                volatile Item* const o = slot(k);
                if (n > 0 && (j0 + n) * BN > S - p.L) {
                    if (b != live_b) {
                        live_b = b;
                        live = 0u;
                        const uint32_t* const mask = p.mask + static_cast<long long>(b) * p.L * p.W;
                        if (p.W <= 4) {  // a lane per draft
                            for (int w = 0; w < p.W; ++w) {
                                const int i = 32 * w + lane;
                                uint32_t any = 0u;
                                for (int x = 0; x < p.W; ++x)
                                    if (i < p.L) any |= __ldg(mask + static_cast<long long>(i) * p.W + x);
                                any = __ballot_sync(0xffffffffu, any != 0u);
                                if (lane == w) live = any;
                            }
                        } else {
#pragma unroll 16
                            for (int i = 0; i < p.L; ++i) {
                                const uint32_t word = lane < p.W ? __ldg(mask + static_cast<long long>(i) * p.W + lane) : 0u;
                                const bool any = __any_sync(0xffffffffu, word != 0u);
                                if (any && lane == (i >> 5)) live |= 1u << (i & 31);
                            }
                        }
                    }
                    o->live[lane] = live;
                }
                if (lane == 0) {
                    o->b = b;
                    o->S = S;
                    o->kvh = kvh;
                    o->mp = mp;
                    o->ng = ng;
                    o->j0 = j0;
                    o->n = n;
                    o->before[0] = before0;
                    o->before[1] = before1;
                    before0 += (n + 1) / 2;
                    before1 += n / 2;
                    if (n > 0 && j0 > 0) from = (seg + kSegCost) / per;
                    if (n > 0 && j0 == 0 && n < ng)  // it ends in a later share
                        crossing = make_int4(b, kvh, mp, (seg + kSegCost + ng - 1) / per);
                    mbar_arrive(bar(kItemFull + k % I));
                }
                __syncwarp();
                if (n == 0 || aborted(abort_flag)) break;
                // on to the next segment
                seg += kSegCost + ng;
                if (seg >= end) continue;
                if (++mp == p.nG) {
                    mp = 0;
                    if (++kvh == p.H_kv) {
                        kvh = 0;
                        do S = seq_len(p, ++b);
                        while (S == 0);
                        ng = key_tiles<BN>(S);
                    }
                }
            }
            if (lane == 0 && rank == 0 && !p.whole) {
                p.split[my_share] = crossing;
                p.join[my_share] = from;
            }
            if (!ok && lane == 0) give_up(p, abort_flag);
        }
        __syncwarp();
    } else {
        // ============================== softmax =======================================
        reg_set<regs(SRC).softmax, launch_regs(SRC)>();
        const int t = (warp - kProd - 4) >> 2, q4 = warp & 3, r = q4 * 32 + lane;  // slot, lane quarter, row
        const uint32_t trow = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
        // How far (log2) a row's scores may rise above its maximum before that moves (and an O
        // relative to it is rescaled): f16 weights end at 2^16, and a sum of bf16 weights times
        // values at 2^128, which leaves N values 2^120 / N.
        constexpr float kSlack = 8.f;
        // f16 weights are taken 2^kLift times as large (O and l are, too): below 2^-14 f16 has
        // steps of 2^-24, so a light key loses 2^-32 of the heaviest one's weight at most.
        constexpr float kLift = F16 ? 7.f : 0.f;
        int xc = 0;  // pieces whose states were joined
        bool ok = true;
        // The end of piece k, with this slot's maximum and sum.  The two slots' states of a row
        // are joined by both warpgroups, 64 dims each (one tile and no halves: A has them all).
        auto finish = [&](int k, float m1, float l1) {
            const volatile Item* const it = slot(k);
            const bool both = HALF || it->n > 1;
            const int m = it->mp * C + rank, rows = p.R - m * BM;
            const bool busy = q4 * 32 < rows, valid = r < rows;
            const int l = static_cast<unsigned>(m * BM + r) % static_cast<unsigned>(p.L);  // draft
            float w0 = 1.f, w1 = 0.f;  // weights of O 0 and O 1 (fp32: of O and the last tile's products)
            if (both) {
                float2* const x = reinterpret_cast<float2*>(smem_raw + M.x) + r;
                ok = xc == 0 || warp_wait(bar(kXFree), (xc - 1) & 1);  // (the last joined piece's are read)
                if (!ok) return false;
                x[t * BM] = make_float2(m1, l1);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kXFull));
                ok = warp_wait(bar(kXFull), xc & 1);
                if (!ok) return false;
                ++xc;
                const float2 a = x[0], e = x[BM];
                const float mm = fmaxf(a.y == 0.f ? neg_inf() : a.x, e.y == 0.f ? neg_inf() : e.x);
                w0 = a.y == 0.f ? 0.f : fast_exp2(a.x - mm);
                w1 = e.y == 0.f ? 0.f : fast_exp2(e.x - mm);
                l1 = (a.y == 0.f ? 0.f : a.y * w0) + (e.y == 0.f ? 0.f : e.y * w1);
                m1 = mm;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kXFree));
                if constexpr (HALF) {
                    const int g = it->before[0] + it->before[1] + it->n - 1, b = 2 * (g & 1);
                    ok = warp_wait(bar(kODone + b), (g >> 1) & 1) && warp_wait(bar(kODone + 1 + b), (g >> 1) & 1);
                    if (!ok) return false;
                } else {
                    const int last = it->n - 1, s = last & 1;
                    const float m0 = reinterpret_cast<const float*>(smem_raw + M.o_max)[(k & 1) * BM + r], mx = s ? e.x : a.x;
                    w0 = m0 == mm ? 1.f : fast_exp2(m0 - mm);
                    w1 = mx == mm ? 1.f : fast_exp2(mx - mm);
                    ok = warp_wait(bar(kODone + s), (it->before[s] + (last >> 1)) & 1);
                    if (!ok) return false;
                    // (behind the arrivals for the tile before, and not before the products that wait for those)
                    if (t == s && lane == 0) mbar_arrive(bar(kTFree));
                }
            } else if (t == 0) {
                ok = warp_wait(bar(kODone), it->before[0] & 1);
                if (!ok) return false;
            }
            const bool full = it->n == it->ng;
            // (a full piece has tail tiles)
            const bool drafted = it->live[l >> 5] >> (l & 31) & 1u;
            const long long row = (static_cast<long long>(it->b) * p.H_kv + it->kvh) * p.R + m * BM + r;
            const long long part = (2ll * blockIdx.x + (it->j0 > 0 ? 0 : 1)) * BM + r;
            if (!full && valid && t == 0) p.part_ml[part] = make_float2(m1, l1);
            if (busy && (both || t == 0)) {
                tc::fence_after_sync();
                const float inv = l1 == 0.f ? 0.f : 1.f / l1;
                // 32 dims a step
#pragma unroll 1
                for (int cc = both ? 2 * t : 0; cc < (both ? 2 * t + 2 : 4); ++cc) {
                    float o[32];
                    __syncwarp();
                    tc::ld32(trow + 256u + cc * 32, o);
                    if (both) {
                        float o1[32];
                        tc::ld32(trow + 384u + cc * 32, o1);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = o[e] * w0 + o1[e] * w1;
                    } else {
                        tc::wait_ld();
                    }
                    if (!valid) continue;
                    if (F32 && full) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = drafted ? o[e] * inv : 0.f;
                        float* const dst = static_cast<float*>(p.out) + row * kD + cc * 32;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            reinterpret_cast<float4*>(dst)[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    } else if (full) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = drafted ? pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv) : 0u;
                        uint16_t* const dst = static_cast<uint16_t*>(p.out) + row * kD + cc * 32;
                        if (p.out32) {  // whole sectors
                            st_global_v8(dst, *reinterpret_cast<const uint32_t(*)[8]>(w));
                            st_global_v8(dst + 16, *reinterpret_cast<const uint32_t(*)[8]>(w + 8));
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                reinterpret_cast<uint4*>(dst)[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
                        }
                    } else if (l1 != 0.f) {
                        float* const dst = p.part_o + part * kD + cc * 32;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            st_global_v8(dst + 8 * e, *reinterpret_cast<const uint32_t(*)[8]>(o + 8 * e));
                    }
                }
                tc::fence_before_sync();
            }
            // O is read: the next piece's first P V may overwrite it
            __syncwarp();
            if (lane == 0) {
                if (both || t == 0) mbar_arrive(bar(kOFree));
                if (!both && t == 0) mbar_arrive(bar(kOFree));  // (for B's warp, which has nothing to read)
                if (HALF) mbar_arrive(bar(kOFree + 1));
            }
            release(k);
            return true;
        };
        for (int k = 0;; ++k) {
            ok = take(k);
            if (!ok) break;
            const int n = slot(k)->n, nk = HALF ? n : (n + 1 - t) >> 1;  // this slot's tiles
            if (n == 0) break;
            const int sc = slot(k)->before[t], g0 = slot(k)->before[0] + slot(k)->before[1];
            const int S = slot(k)->S, first = S - p.L;
            const int m = slot(k)->mp * C + rank;  // query tile
            const int rows = p.R - m * BM;         // of which a tile has at most BM
            const bool busy = q4 * 32 < rows, valid = r < rows;
            const uint32_t* const mask =
                p.mask + (static_cast<long long>(slot(k)->b) * p.L + static_cast<unsigned>(m * BM + r) % static_cast<unsigned>(p.L)) * p.W;
            float c = fmaxf(p.scale_log2, FLT_MIN);  // (scale 0: -inf stays -inf)
            if constexpr (F16) {
                // A takes the rows to f16 (fp32: two parts), the largest value in [2^14, 2^15):
                // 16-bit rows in place, fp32 rows from global memory
                const int buf = q_buf(k);
                float* const down = reinterpret_cast<float*>(smem_raw + M.q_scale) + buf * BM + r;
                if (t == 0) {
                    const uint32_t qrow = base + buf * (QP * kQTile / 2);
                    if constexpr (F32) {
                        // (the products of the last piece in the buffer are done)
                        ok = q_use(k) == 0 || warp_wait(bar(kQEmpty + buf), (q_use(k) - 1) & 1);
                        if (!ok) break;
                        if (busy) {
                            // a row at once, four dims a lane, eight rows on their way (sixteen: registers run out)
                            const long long first_row =
                                (static_cast<long long>(slot(k)->b) * p.H_kv + slot(k)->kvh) * p.R + m * BM + q4 * 32;
                            const float4* const src = reinterpret_cast<const float4*>(p.q + first_row * kD) + lane;
                            const uint32_t at = qrow + (lane >> 4) * p.q_half + (lane & 1) * 8;
#pragma unroll 1
                            for (int r0 = 0; r0 < 32 && q4 * 32 + r0 < rows; r0 += 8) {
                                float4 v[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    v[i] = q4 * 32 + r0 + i < rows ? __ldg(src + (r0 + i) * (kD / 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    // (as bits: the order of numbers above 0)
                                    const float mx = fmax3(fmaxf(fabsf(v[i].x), fabsf(v[i].y)), fabsf(v[i].z), fabsf(v[i].w));
                                    float up, dn;
                                    f16_scale(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx))), up, dn);
                                    uint32_t hi[2], lo[2];
                                    split_f16(make_float2(v[i].x * up, v[i].y * up), hi[0], lo[0]);
                                    split_f16(make_float2(v[i].z * up, v[i].w * up), hi[1], lo[1]);
                                    const int x = q4 * 32 + r0 + i;
                                    const uint32_t to = at + sw128(x, lane >> 1 & 7);
                                    sts64(to, hi[0], hi[1]);
                                    sts64(to + 2 * p.q_half, lo[0], lo[1]);
                                    if (lane == 0) down[x - r] = dn;
                                }
                            }
                        }
                    } else {
                        ok = warp_wait(bar(kQFull + buf), q_use(k) & 1);
                        if (!ok) break;
                        if (busy) {
                            uint4 v[16];
                            float mx = 0.f;
#pragma unroll
                            for (int c = 0; c < 16; ++c) {
                                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                             : "=r"(v[c].x), "=r"(v[c].y), "=r"(v[c].z), "=r"(v[c].w)
                                             : "r"(qrow + (c >> 3) * p.q_half + sw128(r, c & 7)));
                                const float2 f[4] = {bf16x2_to_float2(v[c].x), bf16x2_to_float2(v[c].y),
                                                     bf16x2_to_float2(v[c].z), bf16x2_to_float2(v[c].w)};
#pragma unroll
                                for (int e = 0; e < 4; ++e) mx = fmax3(mx, fabsf(f[e].x), fabsf(f[e].y));
                            }
                            float up, dn;
                            f16_scale(mx, up, dn);
#pragma unroll
                            for (int c = 0; c < 16; ++c) {
                                const float2 f[4] = {bf16x2_to_float2(v[c].x), bf16x2_to_float2(v[c].y),
                                                     bf16x2_to_float2(v[c].z), bf16x2_to_float2(v[c].w)};
                                sts128(qrow + (c >> 3) * p.q_half + sw128(r, c & 7), pack_f16x2(f[0].x * up, f[0].y * up),
                                       pack_f16x2(f[1].x * up, f[1].y * up), pack_f16x2(f[2].x * up, f[2].y * up),
                                       pack_f16x2(f[3].x * up, f[3].y * up));
                            }
                            *down = dn;
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kQReady + buf));
                }
            }
            const int tail = first_tail(S);
            float mrow = neg_inf();
            float2 lsum = make_float2(0.f, 0.f);
            const int j0 = slot(k)->j0;
            for (int j = 0; j < nk; ++j) {
                const int i = HALF ? j : 2 * j + t, jt = j0 + i;  // key tile
                // the places of S, P and their uses before
                const int b = HALF ? (g0 + j) & 1 : 0, use = HALF ? (g0 + j) >> 1 : sc + j;
                uint32_t see[UK / 32];
                if (busy && jt >= tail) {  // this row's bits of the tile, while S is on its way
                    const int x = jt * BN + (HALF ? UK * t : 0) - first;
                    const int w0 = x >> 5, sh = x & 31;  // (floor: words before the drafts are all ones)
                    uint32_t w[UK / 32 + 1];
#pragma unroll
                    for (int e = 0; e < UK / 32 + 1; ++e) {
                        const int wi = w0 + e;
                        w[e] = wi < 0 ? 0xffffffffu : wi < p.W ? __ldg(mask + wi) & slot(k)->live[wi] : 0u;
                    }
#pragma unroll
                    for (int e = 0; e < UK / 32; ++e) see[e] = __funnelshift_r(w[e], w[e + 1], sh);
                }
                ok = warp_wait(bar(kSFull + (HALF ? b : t)), use & 1);
                if (!ok || aborted(abort_flag)) break;
                if constexpr (SRC == kF32) {  // the scales of this tile's V
                    const int tile = g0 + i;
                    ok = warp_wait(bar(kVScale + (tile & 3)), (tile >> 2) & 1);
                    if (!ok) break;
                }
                if constexpr (F16) {
                    if (j == 0) {  // (S is there, so this use of the buffer was announced, and none after it)
                        const int buf = q_buf(k);
                        ok = warp_wait(bar(kQReady + buf), q_use(k) & 1);
                        if (!ok) break;
                        if (busy)
                            c = fmaxf(reinterpret_cast<const float*>(smem_raw + M.q_scale)[buf * BM + r] * p.scale_log2, FLT_MIN);
                    }
                }
                if (busy) {
                    tc::fence_after_sync();
                    const uint32_t st = trow + (HALF ? 128u * b + UK * t : 128u * t);
                    float2 ts = make_float2(0.f, 0.f);
                    float mx = neg_inf(), alpha = 1.f;
                    // 32 scores of a tail tile, those that this row does not see masked
                    auto hide = [&](float (&x)[32], int cc) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(see[cc] >> e & 1u)) x[e] = neg_inf();
                    };
                    // the largest of 32 scores and mx
                    auto largest = [&](const float (&x)[32]) {
                        float a = fmax3(x[0], x[1], mx), b = x[2];
#pragma unroll
                        for (int e = 3; e < 31; e += 4) {
                            a = fmax3(a, x[e], x[e + 1]);
                            b = fmax3(b, x[e + 2], x[e + 3]);
                        }
                        mx = fmax3(a, b, x[31]);
                    };
                    // their weights against the maximum mu
                    auto weights = [&](float (&x)[32], uint32_t* w, float mu) {
                        const float2 c2 = make_float2(c, c), nm2 = make_float2(-mu, -mu);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 y = __ffma2_rn(make_float2(x[2 * i], x[2 * i + 1]), c2, nm2);
                            const float2 ex = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                            w[i] = F16 ? pack_f16x2(ex.x, ex.y) : pack_bf16x2(ex.x, ex.y);
                            ts = __fadd2_rn(ts, ex);
                        }
                    };
                    // the tile's maximum from all of S; true where the row's moved
                    auto maximum = [&]() {
#pragma unroll
                        for (int cc = 0; cc < UK / 32; ++cc) {
                            float x[32];
                            tc::ld32(st + cc * 32, x);
                            tc::wait_ld();
                            if (jt >= tail) hide(x, cc);
                            largest(x);
                        }
                        const float mt = mx * c;
                        const bool grow = valid && mt > mrow;  // (other rows hold anything)
                        if (grow) {
                            alpha = fast_exp2(mrow - mt);  // 2^-inf = 0 at the start
                            mrow = mt;
                        }
                        return __any_sync(0xffffffffu, grow);
                    };
                    // O is rescaled once this slot's previous P V is done
                    auto rescale = [&]() {
                        const int g = g0 + j - 1;
                        if (!warp_wait(bar(kODone + t + (HALF ? 2 * (g & 1) : 0)), (HALF ? g >> 1 : sc + j - 1) & 1)) return false;
                        tc::fence_after_sync();
#pragma unroll 1
                        for (int cc = 0; cc < 4; ++cc) {
                            float o[32];
                            tc::ld32(trow + 256u + 128u * t + cc * 32, o);
                            tc::wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= alpha;
                            tc::st32(trow + 256u + 128u * t + cc * 32, o);
                        }
                        tc::wait_st();
                        return true;
                    };
                    // P goes over the first columns of its S
                    if constexpr (F32) {
                        // Two parts of P do not fit the registers beside S: the masked scores, scaled
                        // to powers of two, go back over S, and then 32 keys' P over their own (all
                        // done twice, from S as it was, the second 32 keys unrolled: fp32 pages, 256
                        // rows, 192 us for 172, fp32 queries over 4 bits 57 for 51).  fp32 pages: V's
                        // rows were scaled by 2^v, so P is 2^(score - v - maximum), the maximum that
                        // of score - v, and the sum adds P 2^v: the weights relative to that maximum.
                        const float4* const k_scale = reinterpret_cast<const float4*>(smem_raw + M.kv_scale) + ((g0 + i) & 7) * (BN / 4);
                        const float4* const v_scale = reinterpret_cast<const float4*>(smem_raw + M.kv_scale) + (8 + ((g0 + i) & 3)) * (BN / 4);
#pragma unroll
                        for (int cc = 0; cc < BN / 32; ++cc) {
                            float x[32];
                            tc::ld32(st + cc * 32, x);
                            tc::wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                float4 kf = make_float4(c, c, c, c), off = make_float4(0.f, 0.f, 0.f, 0.f);
                                if constexpr (SRC == kF32) {
                                    const float4 ks = k_scale[cc * 8 + e / 4];
                                    kf = make_float4(c * ks.x, c * ks.y, c * ks.z, c * ks.w);
                                    off = v_scale[cc * 8 + e / 4];
                                }
                                x[e] = fmaf(x[e], kf.x, -off.x);
                                x[e + 1] = fmaf(x[e + 1], kf.y, -off.y);
                                x[e + 2] = fmaf(x[e + 2], kf.z, -off.z);
                                x[e + 3] = fmaf(x[e + 3], kf.w, -off.w);
                            }
                            if (jt >= tail) {
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (!(see[cc] >> e & 1u)) x[e] = neg_inf();
                            }
                            tc::st32(st + cc * 32, x);
#pragma unroll
                            for (int e = 0; e < 32; e += 2) mx = fmax3(mx, x[e], x[e + 1]);
                        }
                        tc::wait_st();
                        const bool grow = valid && mx > mrow + kSlack;
                        if (grow) {
                            alpha = fast_exp2(mrow - mx);  // 2^-inf = 0 at the start
                            mrow = mx;
                        }
                        const float mu = mrow == neg_inf() ? 0.f : mrow - kLift;
#pragma unroll 1  // (registers)
                        for (int cc = 0; cc < BN / 32; ++cc) {
                            float x[32];
                            tc::ld32(st + cc * 32, x);
                            tc::wait_ld();
                            uint32_t w[32];  // 16 of the high parts, 16 of the low ones
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 ex = make_float2(fast_exp2(x[2 * i] - mu), fast_exp2(x[2 * i + 1] - mu));
                                split_f16(ex, w[i], w[16 + i]);
                                if constexpr (SRC == kF32) {
                                    const float2 back = reinterpret_cast<const float2*>(v_scale + BN)[cc * 16 + i];
                                    ts = __ffma2_rn(ex, back, ts);
                                } else {
                                    ts = __fadd2_rn(ts, ex);
                                }
                            }
                            tc::st32(st + cc * 32, w);
                        }
                    } else {
                        // Against the maximum so far: no weight waits for the scores behind it.  Only
                        // where that was too low by 2^kSlack (or there was none) is the tile done
                        // again, with its own maximum.
                        uint32_t pw[UK / 2];
                        bool again = true;
                        if (j > 0) {
                            const float mu = mrow == neg_inf() ? 0.f : mrow - kLift;
                            float x[UK / 32][32];
#pragma unroll
                            for (int cc = 0; cc < UK / 32; ++cc) tc::ld32(st + cc * 32, x[cc]);
                            tc::wait_ld();
                            if (jt >= tail) {
#pragma unroll
                                for (int cc = 0; cc < UK / 32; ++cc) hide(x[cc], cc);
                            }
#pragma unroll
                            for (int cc = 0; cc < UK / 32; ++cc) {
                                largest(x[cc]);
                                weights(x[cc], pw + 16 * cc, mu);
                            }
                            again = __any_sync(0xffffffffu, valid && mx * c > mrow + kSlack);
                        }
                        if (again) {
                            mx = neg_inf();
                            if (maximum() && j > 0) {
                                ok = rescale();
                                if (!ok) break;
                            }
                            ts = make_float2(0.f, 0.f);
                            const float mu = mrow == neg_inf() ? 0.f : mrow - kLift;
#pragma unroll
                            for (int cc = 0; cc < UK / 32; ++cc) {
                                float x[32];
                                tc::ld32(st + cc * 32, x);
                                tc::wait_ld();
                                if (jt >= tail) hide(x, cc);
                                weights(x, pw + 16 * cc, mu);
                            }
                        }
                        tc::st32(st, pw);
                    }
                    lsum.x = lsum.x * alpha + ts.x;
                    lsum.y = lsum.y * alpha + ts.y;
                    tc::wait_st();
                    tc::fence_before_sync();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kPFull + t + 2 * b));
                if constexpr (!HALF) {
                    // The first tile's products are O.  The others' are added to it here, one tile after
                    // the other, but for the last tile's, which are where the piece ends.
                    float* const o_max = reinterpret_cast<float*>(smem_raw + M.o_max) + (k & 1) * BM + r;
                    const bool here = i > 0 && i < n - 1;
                    if (here) ok = warp_wait(bar(kODone + t), use & 1) && warp_wait(bar(kTFree), (g0 + i - 1) & 1);
                    if (!ok) break;
                    if (busy && i == 0) *o_max = mrow;
                    if (busy && here) {
                        tc::fence_after_sync();
                        const float m0 = *o_max, mm = fmaxf(m0, mrow);
                        const float w0 = m0 == mm ? 1.f : fast_exp2(m0 - mm), w1 = mrow == mm ? 1.f : fast_exp2(mrow - mm);
#pragma unroll 1
                        for (int cc = 0; cc < 4; ++cc) {
                            float o[32], x[32];
                            tc::ld32(trow + 256u + cc * 32, o);
                            tc::ld32(trow + 384u + cc * 32, x);
                            tc::wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = fmaf(x[e], w1, o[e] * w0);
                            tc::st32(trow + 256u + cc * 32, o);
                        }
                        *o_max = mm;
                        tc::wait_st();
                        tc::fence_before_sync();
                    }
                    __syncwarp();
                    if (lane == 0 && (i == 0 || here)) mbar_arrive(bar(kTFree));
                }
            }
            if (!ok || aborted(abort_flag)) break;
            ok = finish(k, mrow, lsum.x + lsum.y);
            if (!ok) break;
        }
        if (!ok && lane == 0) give_up(p, abort_flag);
    }

    // ---- tear-down: free TMEM once every role is done ---------------------------
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kProd) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

// Rows r .. r + ROWS - 1 of the segment that starts in share c and ends in share sp.w, its
// partial states U at a time: four loads in flight.
template <bool F32, int ROWS, int U>
__device__ __forceinline__ void merge_rows(const TileParams& p, int C, const int4 sp, int c, int r) {
    const int lane = threadIdx.x & 31;
    const int in_head = sp.z * C * BM + r;
    if (r >= C * BM || in_head >= p.R) return;
    uint32_t drafted[ROWS];  // a word of the row's mask
    float M[ROWS], sum[ROWS];
    float4 acc[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const uint32_t* const m = p.mask + (static_cast<long long>(sp.x) * p.L + (in_head + i) % p.L) * p.W;
        drafted[i] = lane < p.W ? __ldg(m + lane) : 0u;
        M[i] = neg_inf();
        sum[i] = 0.f;
        acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int k = c; k <= sp.w; k += U) {
        float2 v[U][ROWS];
        float4 x[U][ROWS];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                v[u][i] = make_float2(neg_inf(), 0.f);
                if (k + u > sp.w || in_head + i >= p.R) continue;
                const int cta = (k + u) * C + (r + i) / BM;
                const long long slot = (2ll * cta + (k + u == c ? 1 : 0)) * BM + (r + i) % BM;
                v[u][i] = p.part_ml[slot];
                x[u][i] = *reinterpret_cast<const float4*>(p.part_o + slot * kD + 4 * lane);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                if (v[u][i].y == 0.f) continue;  // no key (x was not written)
                const float mx = fmaxf(M[i], v[u][i].x), a = fast_exp2(M[i] - mx), b = fast_exp2(v[u][i].x - mx);
                M[i] = mx;
                sum[i] = sum[i] * a + v[u][i].y * b;
                acc[i].x = acc[i].x * a + x[u][i].x * b;
                acc[i].y = acc[i].y * a + x[u][i].y * b;
                acc[i].z = acc[i].z * a + x[u][i].z * b;
                acc[i].w = acc[i].w * a + x[u][i].w * b;
            }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const bool live = __any_sync(0xffffffffu, drafted[i] != 0u);
        if (in_head + i >= p.R) continue;
        const float inv = sum[i] == 0.f ? 0.f : 1.f / sum[i];  // (0: a row without keys; NaN stays)
        const long long row = (static_cast<long long>(sp.x) * p.H_kv + sp.y) * p.R + in_head + i;
        float4 o = make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv);
        if (!live) o = make_float4(0.f, 0.f, 0.f, 0.f);
        if constexpr (F32)
            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * kD + 4 * lane) = o;
        else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * kD + 4 * lane) =
                make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
    }
}

// Merges the partial states of the segments that cross shares.  The ny CTAs of a share take
// part in the segment that comes into it, so one cut into many pieces has as many CTAs, a
// warp a row of it (one sequence of 16000 keys: 33 us in all with the CTAs of its first share
// alone, 27 with all).  What it takes is its launch and L2's latency: 4 to 7 us of a call.
constexpr int kMergeRows = 2;
template <bool F32>
__global__ void __launch_bounds__(256, 3) tree_merge_kernel(const TileParams p, int ny, int C) {
    const int k = static_cast<int>(blockIdx.x) / ny, y = static_cast<int>(blockIdx.x) - k * ny;
    pdl_wait_primary();
    const int c = p.join[k];
    if (c < 0) return;
    const int4 sp = p.split[c];
    if (sp.x < 0) return;  // (a share that gave up)
    const int groups = sp.w - c, at = ((k - c - 1) * ny + y) * 8 + static_cast<int>(threadIdx.x >> 5);
    if (groups == 1) merge_rows<F32, kMergeRows, 2>(p, C, sp, c, at * kMergeRows);
    else merge_rows<F32, 1, 4>(p, C, sp, c, at);
}

struct TilePlan {
    size_t split_off, join_off, ml_off, o_off, total;
};

// (the same for every shape)
TilePlan plan(int sm_count) {
    TilePlan t;
    const size_t states = 2ull * sm_count * BM;
    t.split_off = kFlagBytes;
    t.join_off = t.split_off + 16ull * sm_count;
    t.ml_off = align_up(t.join_off + 4ull * sm_count, 256);
    t.o_off = align_up(t.ml_off + states * 8, 256);
    t.total = t.o_off + states * kD * 4;
    return t;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
        else
            cudaGetLastError();
    });
    return fn;
}

// 4-D map of a pool: 64 dims, 8 rows, 2 halves of the dims, groups of 8 rows; boxes of
// box_rows rows land as [8 rows][half][row][64 dims], 128-byte swizzle.
bool make_pool_map(CUtensorMap* map, const void* ptr, long long rows, int box_rows) {
    const auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {64, 8, 2, static_cast<cuuint64_t>(rows / 8)};
    const cuuint64_t strides[3] = {kD * 2, kD, 8 * kD * 2};
    const cuuint32_t box[4] = {64, 8, 2, static_cast<cuuint32_t>(box_rows / 8)};
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, steps,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <Source SRC, int C>
pa_status launch_tiles(TileParams p, const CUtensorMap* maps, const TreeCall& c, int* shares) {
    constexpr int bytes = smem(SRC).total;
    static int ready[64] = {0};  // per device
    if (!ready[c.dev.device]) {
        if (cudaFuncSetAttribute(tree_tile_kernel<SRC, C>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
            return PA_ERR_CUDA;
        // the roles' registers come out of what the launch has
        cudaFuncAttributes at;
        if (cudaFuncGetAttributes(&at, tree_tile_kernel<SRC, C>) != cudaSuccess) return PA_ERR_CUDA;
        if (at.numRegs != launch_regs(SRC)) return PA_ERR_UNSUPPORTED;
        ready[c.dev.device] = 1;
    }
    *shares = c.dev.sm_count / C;
    if (*shares < 1) return PA_ERR_UNSUPPORTED;
    const long long segs = static_cast<long long>(p.B) * p.H_kv * p.nG;
    p.whole = segs <= *shares && p.max_S <= (4 * segs < *shares ? kWholeFew : kWholeMany) * keys(SRC);
    if (p.whole) *shares = static_cast<int>(segs);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(*shares * C));
    cfg.blockDim = dim3(threads(SRC));
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = c.stream;
    if (cudaLaunchKernelEx(&cfg, tree_tile_kernel<SRC, C>, p, maps[0], maps[1], maps[2]) != cudaSuccess) return PA_ERR_CUDA;
    if (p.whole) *shares = 0;
    return PA_OK;
}

int gcd_int(int a, int b) {
    while (b) {
        const int t = a % b;
        a = b;
        b = t;
    }
    return a;
}

}  // namespace

bool tree_supported(const pa_shape& sh) {
    if (sh.L > kTreeMax || static_cast<long long>(sh.B) * sh.H_q * sh.L >= INT_MAX) return false;
    const long long R = static_cast<long long>(sh.H_q / sh.H_kv) * sh.L;
    const long long cap = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    // costs are counted in an int
    return static_cast<long long>(sh.B) * sh.H_kv * ((R + BM - 1) / BM) * (cap / keys(kF32) + 1 + kSegCost) < INT_MAX / 2;
}

size_t tree_workspace_bytes(int sm_count) { return plan(sm_count).total; }

pa_status tree_launch(const TreeCall& c) {
    const pa_shape& sh = c.sh;
    if (c.dev.smem_optin < 232448) return PA_ERR_UNSUPPORTED;
    const TilePlan t = plan(c.dev.sm_count);
    uint8_t* const ws = static_cast<uint8_t*>(c.ws);
    TileParams p;
    p.kc = static_cast<const uint8_t*>(c.kc);
    p.ks = static_cast<const uint8_t*>(c.ks);
    p.vc = static_cast<const uint8_t*>(c.vc);
    p.vs = static_cast<const uint8_t*>(c.vs);
    p.bt = c.bt;
    p.ctx = c.ctx;
    p.mask = c.mask;
    p.q = static_cast<const float*>(c.q);
    p.out = c.out;
    p.flag = reinterpret_cast<uint32_t*>(ws);
    p.part_ml = reinterpret_cast<float2*>(ws + t.ml_off);
    p.part_o = reinterpret_cast<float*>(ws + t.o_off);
    p.split = reinterpret_cast<int4*>(ws + t.split_off);
    p.join = reinterpret_cast<int*>(ws + t.join_off);
    p.B = sh.B;
    p.H_kv = sh.H_kv;
    p.R = sh.H_q / sh.H_kv * sh.L;
    p.L = sh.L;
    p.W = tree_words(sh.L);
    p.num_pages = sh.num_pages;
    p.ps = sh.page_size;
    p.max_npg = sh.max_pages_per_seq;
    p.pool_rows = sh.num_pages * sh.H_kv * sh.page_size;
    p.q_box = std::min(BM, (p.R + 7) / 8 * 8);
    p.q_bufs = p.q_box <= BM / 2 ? 2 : 1;
    p.q_half = kQTile / 2 / p.q_bufs;
    const bool f32 = sh.dtype == PA_F32;
    p.max_S = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    p.scale_log2 = c.scale * 1.4426950408889634f;
    p.out32 = reinterpret_cast<uintptr_t>(c.out) % 32 == 0;
    const bool tma = !f32 && !c.ks && sh.page_size % 8 == 0;
    // Two query tiles side by side read K and V from HBM once (a tile alone at a time, in turn:
    // 252 rows 98 us, in pairs 76; 256 rows 178 and 136; 1020 rows 180 and 162; an odd number
    // leaves a CTA of the last pair without rows: 260 rows 72 and 79).
    const int nM = (p.R + BM - 1) / BM, C = tma && nM > 1 ? 2 : 1;
    p.nG = (nM + C - 1) / C;
    p.box = gcd_int(sh.page_size, keys(kTma));
    CUtensorMap maps[3] = {};
    if (!f32 && !make_map(&maps[0], c.q, static_cast<long long>(sh.B) * sh.H_q * sh.L, p.q_box)) return PA_ERR_CUDA;
    maps[1] = maps[2] = maps[0];
    if (tma && (!make_pool_map(&maps[1], c.kc, p.pool_rows, p.box) || !make_pool_map(&maps[2], c.vc, p.pool_rows, p.box)))
        return PA_ERR_CUDA;
    int shares = 0;
    const pa_status st = f32     ? c.ks ? launch_tiles<kQ4F, 1>(p, maps, c, &shares) : launch_tiles<kF32, 1>(p, maps, c, &shares)
                         : c.ks  ? launch_tiles<kQ4, 1>(p, maps, c, &shares)
                         : !tma  ? launch_tiles<kCopy, 1>(p, maps, c, &shares)
                         : C > 1 ? launch_tiles<kTma, 2>(p, maps, c, &shares)
                                 : launch_tiles<kTma, 1>(p, maps, c, &shares);
    if (st != PA_OK || shares == 0) return st;  // (0: nothing to merge)
    const int ny = (std::min(p.R, C * BM) + 8 * kMergeRows - 1) / (8 * kMergeRows);
    return launch_dependent(f32 ? tree_merge_kernel<true> : tree_merge_kernel<false>,
                            dim3(static_cast<unsigned>(shares * ny)), 256, 0, c.stream, p, ny, C)
               ? PA_OK
               : PA_ERR_CUDA;
}

}  // namespace pa
