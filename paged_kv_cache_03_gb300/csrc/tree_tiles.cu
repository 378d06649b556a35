// tree_tiles.cu -- attention of drafted trees for bf16 queries on tcgen05 tensor cores,
// over bf16 and 4-bit pages.
//
// The rows of a (sequence, kv head), r = (query head of the group, draft l), are R = G L
// consecutive rows of the query, cut into tiles of 128.  All of them see every position
// before the drafts, so a key tile of 128 needs no mask unless it holds drafts or lies at
// the end ("tail"); there a row's 128 bits come out of its words of the tree's mask.
//   S = Q K^T,  P = 2^(scale S - m),  O += P V,  with the running maximum m and sum l
// per row; O / l at the end.  bf16 pages: P rounded to bf16, l adds the rounded ones.
// 4-bit pages: K and V dequantised to f16 on chip (exact), Q scaled by a power of two
// into f16's range (exact), P rounded to f16 (2^-11).
//
// Layout on GB300: one CTA per SM, four warpgroups.
//   * A segment is a pair of query tiles (or a lone one) of one (sequence, kv head) over
//     all its key tiles.  The key tiles of all segments are cut into equal shares, one per
//     CTA, so ragged contexts leave no SM idle; a segment that crosses shares leaves fp32
//     partial states that tree_merge_kernel joins.
//   * A job is one key tile for one query tile; job i uses S, P and O of slot t = i & 1.
//     A pair takes jobs (A, key tile 0), (B, 0), (A, 1), ...; a lone tile takes its key
//     tiles in turn in both slots, each with its own m, l and O, which A joins at the end.
//     So both softmax warpgroups work in either case, one on each slot, and the MMA warp
//     issues P V of job i, then Q K^T of job i + 2.
//   * Warps 0-3 bring K and V into two-slot rings in the 128-byte swizzle that the MMA
//     reads: one lane per page box by TMA (bf16, pages of a multiple of 8 slots), 16-byte
//     asynchronous copies (other page sizes), or 4-bit rows dequantised on the way.
//   * Warp 7 publishes the pieces of segments in a ring of four slots, with the bits of
//     the slots that hold drafts, and loads the query tiles by TMA.
//   * Value rows that nobody sees (behind the context, slots without a draft) may hold
//     NaN, and 0 * NaN is NaN: copies leave zeros there, and behind TMA warp 1 zeroes them
//     before the tile is announced.
//   * All waits are bounded; on a timeout the CTA records PA_FLAG_TIMEOUT, frees its TMEM
//     and exits.
#include <algorithm>
#include <cfloat>
#include <climits>

#include "ptx.cuh"
#include "stage.cuh"
#include "tc.cuh"
#include "tree.h"

namespace pa {
namespace {

constexpr int kD = kHeadDim;
constexpr int BM = 128, BN = 128;  // query rows and keys of a tile
constexpr int kThreads = 512;
constexpr uint32_t kTmemCols = 512;  // S of slot t at 128 t, O at 256 + 128 t
constexpr float kLazyRescaleLog2 = 8.0f;
// What a segment's query load, first softmax and epilogue cost, in key tiles: the
// shares count it, or CTAs with many short segments would finish last.
constexpr int kSegCost = 3;
constexpr int kMinPer = 8;  // least cost of a share
constexpr int kHalf = kStageHalf;  // 128 rows x 64 values (one swizzled column block)
constexpr int kTile = 2 * kHalf;
constexpr int kOffQ = 0, kOffK = 2 * kTile, kOffV = 4 * kTile, kOffBar = 6 * kTile;
enum Bar {
    kQFull = 0,     // + buffer: the query tiles are there (4 bit: as they are)
    kQReady = 2,    // + buffer: ... in f16 (4 bit)
    kQEmpty = 4,    // every Q K^T of a piece is done
    kKFull = 5,     // + slot
    kKEmpty = 7,    // + slot
    kVFull = 9,     // + slot
    kVEmpty = 11,   // + slot
    kVTail = 13,    // + slot: a tail tile's values are there, not yet cleaned
    kSFull = 15,    // + t
    kPFull = 17,    // + t
    kODone = 19,    // + t
    kOFree = 21,    // + t: the epilogue has read O
    kXFull = 23,    // + slot: B's max and sum (lone tile)
    kItemFull = 25,   // + slot
    kItemEmpty = 29,  // + slot
    kMmaDone = 33,
    kNumBars = 34
};
constexpr int kItemBytes = 256;
constexpr int kOffItems = kOffBar + kNumBars * 8;
constexpr int kOffTmemSlot = kOffItems + 4 * kItemBytes;
constexpr int kOffAbort = kOffTmemSlot + 8;
constexpr int kOffX = kOffAbort + 8;             // [2][128] max and sum of B's rows
constexpr int kOffQScale = kOffX + 2 * BM * 8;   // 4 bit: [2][128] the inverse of a row's scale
constexpr int kOffRaw = kOffQScale + 2 * BM * 4; // 4 bit: [warp][K, V] rows on their way
static_assert(kOffItems % 16 == 0 && kOffRaw % 16 == 0, "16-byte copies");
enum Source { kTma, kCopy, kQ4 };
constexpr int smem_bytes(Source s) { return (s == kQ4 ? kOffRaw + 4 * 2 * kRawStage : kOffQScale) + 1024; }

struct TileParams {
    const uint8_t *kc, *ks, *vc, *vs;  // codes or bf16 rows, scales
    const int32_t* bt;
    const int32_t* ctx;
    const uint32_t* mask;
    uint16_t* out;
    uint32_t* flag;
    float2* part_ml;  // [2 per CTA][tile][128]: max, sum
    float* part_o;    // [2 per CTA][tile][128][D]
    int4* split;      // per CTA: the segment that starts in its share and ends in a later one
    int B, H_kv, R, L, W, nM, nPairs, num_pages, ps, max_npg;
    int pool_rows, box, q_box;  // rows of the pool, of a K/V box, of a query box
    long long max_S;
    float scale_log2;
    int out32;  // the output is 32-byte aligned
};

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// Length of a sequence, 0 for one that breaks the contract.
__device__ __forceinline__ int seq_len(const TileParams& p, int b) {
    const int S = __ldg(p.ctx + b);
    return S < p.L || static_cast<long long>(S) > p.max_S ? 0 : S;
}
__device__ __forceinline__ int key_tiles(int S) { return (S + BN - 1) / BN; }
__device__ __forceinline__ int seq_cost(const TileParams& p, int S) {
    return S == 0 ? 0 : p.H_kv * p.nPairs * (kSegCost + key_tiles(S));
}

// A published piece: key tiles j0 .. j0 + n - 1 of its ng, for nt query tiles.  Slot k & 3
// holds piece k from kItemFull to kItemEmpty.
struct Item {
    int b, S, kvh, mp, ng, j0, n, nt;  // n = 0: no more
    int jobs[2];    // jobs of slot t
    int before[2];  // ... in earlier pieces
    uint32_t live[32];  // slots that hold a draft (pieces with tail tiles)
};
static_assert(sizeof(Item) <= kItemBytes, "item slot");

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}
__device__ __forceinline__ bool aborted(volatile int* f) { return __any_sync(0xffffffffu, *f != 0); }
__device__ __forceinline__ void give_up(const TileParams& p, volatile int* f) {
    *f = 1;
    atomicOr(p.flag, PA_FLAG_TIMEOUT);
}

constexpr uint32_t idesc(bool f16, int a_mn, int b_mn) {
    return tc::idesc_bf16(BM, BN, a_mn, b_mn) & ~(f16 ? (1u << 7) | (1u << 10) : 0u);
}

template <int N>
__device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// MULTI: more than one query tile per (sequence, kv head).  Without it the two query
// buffers take the pieces in turn.
template <Source SRC, bool MULTI>
__global__ void __launch_bounds__(kThreads, 1)
    tree_tile_kernel(const TileParams p, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
    constexpr bool Q4 = SRC == kQ4;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int share[4];  // all units, units per share, first sequence, its first unit
    __shared__ int sums[kThreads / 32];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* const sbase = smem_raw + (base - raw);
    const uint32_t bar0 = base + kOffBar;
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(sbase + kOffAbort);
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(sbase + kOffTmemSlot);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();

    // ---- set-up ----------------------------------------------------------------
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(kQFull + s), 1);
            mbar_init(bar(kQReady + s), MULTI ? 8 : 4);
            mbar_init(bar(kKFull + s), SRC == kTma ? 1 : 4);
            mbar_init(bar(kKEmpty + s), 1);
            mbar_init(bar(kVFull + s), SRC == kTma ? 1 : 4);
            mbar_init(bar(kVEmpty + s), 1);
            mbar_init(bar(kVTail + s), 1);
            mbar_init(bar(kSFull + s), 1);
            mbar_init(bar(kPFull + s), 4);
            mbar_init(bar(kODone + s), 1);
            mbar_init(bar(kOFree + s), 4);
            mbar_init(bar(kXFull + s), 4);
        }
        mbar_init(bar(kQEmpty), 1);
        mbar_init(bar(kMmaDone), 1);
        for (int s = 0; s < 4; ++s) {
            mbar_init(bar(kItemFull + s), 1);
            // K/V warps, the MMA thread, softmax warps
            mbar_init(bar(kItemEmpty + s), (SRC == kTma ? 2 : 4) + 1 + 8);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 4) {
        tc::tmem_alloc(base + kOffTmemSlot, kTmemCols);
        tc::tmem_relinquish();
    }
    // ---- this CTA's share --------------------------------------------------------
    {
        int mine = 0, v = 0;
        for (int b = tid; b < p.B; b += kThreads) {
            const int n = seq_cost(p, seq_len(p, b));
            if (b == tid) mine = n;
            v += n;
        }
        v = __reduce_add_sync(0xffffffffu, v);
        if (lane == 0) sums[warp] = v;
        __syncthreads();
        int total = 0;
        for (int w = 0; w < kThreads / 32; ++w) total += sums[w];
        const int per = max((total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x), kMinPer);
        const int u = static_cast<int>(blockIdx.x) * per;
        if (tid == 0) {
            share[0] = total;
            share[1] = per;
        }
        int carry = 0;
        for (int b0 = 0; b0 < p.B; b0 += kThreads) {
            const int b = b0 + tid;
            int x = mine;
            if (b0 > 0) x = b < p.B ? seq_cost(p, seq_len(p, b)) : 0;
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
        // sequences that break the contract: zero rows
        for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
            if (seq_len(p, b) > 0) continue;
            if (tid == 0) atomicOr(p.flag, PA_FLAG_BAD_CONTEXT);
            const long long rows = static_cast<long long>(p.H_kv) * p.R;
            uint4* const o = reinterpret_cast<uint4*>(p.out + b * rows * kD);
            for (long long i = tid; i < rows * (kD / 8); i += kThreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    auto slot = [&](int k) { return reinterpret_cast<volatile Item*>(sbase + kOffItems + kItemBytes * (k & 3)); };
    auto take = [&](int k) { return warp_wait(bar(kItemFull + (k & 3)), (k >> 2) & 1); };  // a whole warp
    auto release = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kItemEmpty + (k & 3)));
    };
    // key tiles of a piece from this one on hold drafts or the context's end
    auto first_tail = [&](int S) { return (S - p.L) / BN; };

    if (warp < 4) {
        // ========================= K/V producers ==================================
        reg_dec<72>();
        bool ok = true;
        if constexpr (SRC == kTma) {
            if (warp == 0) {
                const uint64_t policy = p.nPairs == 1 ? l2_policy_evict_first() : l2_policy_evict_last();
                const int nbox = BN / p.box;
                bool bad_page = false;
                int g = 0;  // tiles so far
                for (int k = 0;; ++k) {
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
                    for (int j = j0; j < j0 + n; ++j, ++g) {
                        const int s = g & 1, key = j * BN + lane * p.box;
                        const bool mine = lane < nbox && key < S;
                        const bool good = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages);
                        bad_page |= mine && !good;
                        // (a row behind the pool reads as zeros)
                        const int row = good ? (page * p.H_kv + kvh) * p.ps + key % p.ps : p.pool_rows;
                        const uint32_t bytes = static_cast<uint32_t>(min(nbox, (S - j * BN + p.box - 1) / p.box)) * p.box * 256u;
                        if (j + 1 < j0 + n) page = page_of(j + 1);
                        if (g >= 2 && !warp_wait(bar(kKEmpty + s), ((g >> 1) - 1) & 1)) {
                            ok = false;
                            break;
                        }
                        if (aborted(abort_flag)) break;
                        if (lane == 0) mbar_arrive_expect_tx(bar(kKFull + s), bytes);
                        __syncwarp();
                        if (mine) {
                            const uint32_t dst = base + kOffK + s * kTile + lane * p.box * 128;
                            tc::tma_load_2d(dst, &kmap, 0, row, bar(kKFull + s), policy);
                            tc::tma_load_2d(dst + kHalf, &kmap, 64, row, bar(kKFull + s), policy);
                        }
                        if (g >= 2 && !warp_wait(bar(kVEmpty + s), ((g >> 1) - 1) & 1)) {
                            ok = false;
                            break;
                        }
                        if (aborted(abort_flag)) break;
                        const uint32_t vbar = bar((j >= tail ? kVTail : kVFull) + s);
                        if (lane == 0) mbar_arrive_expect_tx(vbar, bytes);
                        __syncwarp();
                        if (mine) {
                            const uint32_t dst = base + kOffV + s * kTile + lane * p.box * 128;
                            tc::tma_load_2d(dst, &vmap, 0, row, vbar, policy);
                            tc::tma_load_2d(dst + kHalf, &vmap, 64, row, vbar, policy);
                        }
                    }
                    if (!ok || aborted(abort_flag)) break;
                }
                // no copy may land after the CTA's shared memory is gone: the last tiles'
                for (int s = 0; s < 2; ++s)
                    if (g > s) {
                        const int u = (g - 1 - s) & 1, x = (g - 1 - s) >> 1;  // tile g - 1 - s, use x of its slot
                        if (!warp_wait(bar(kKFull + u), x & 1) || !warp_wait(bar(kVFull + u), x & 1)) ok = false;
                    }
                if (__any_sync(0xffffffffu, bad_page) && lane == 0) atomicOr(p.flag, PA_FLAG_BAD_PAGE);
            } else if (warp == 1) {
                // value rows of tail tiles that nobody sees
                int g = 0, tails[2] = {0, 0};
                for (int k = 0;; ++k) {
                    ok = take(k);
                    if (!ok) break;
                    const int n = slot(k)->n, j0 = slot(k)->j0, S = slot(k)->S, first = S - p.L, tail = first_tail(S);
                    for (int j = max(j0, tail); j < j0 + n && ok; ++j) {
                        const int s = (g + j - j0) & 1;
                        ok = warp_wait(bar(kVTail + s), (s ? tails[1] : tails[0]) & 1);
                        if (!ok) break;
                        if (s) ++tails[1];
                        else ++tails[0];
#pragma unroll 1
                        for (int r = lane; r < BN; r += 32) {
                            const int x = j * BN + r - first;  // draft
                            if (x < 0 || (x < p.L && (slot(k)->live[x >> 5] >> (x & 31) & 1u))) continue;
                            const uint32_t at = base + kOffV + s * kTile + r * 128;
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                sts128(at + 16 * c, 0u, 0u, 0u, 0u);
                                sts128(at + kHalf + 16 * c, 0u, 0u, 0u, 0u);
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(kVFull + s));
                    }
                    g += n;
                    release(k);
                    if (!ok || n == 0 || aborted(abort_flag)) break;
                }
            }
        } else {
            // pool rows of the next tile, lane 8 i + r: key 32 i + 8 warp + r; -1 where
            // nobody sees the key
            int page = 0, in_page = -1, row_base = 0;
            bool bad_page = false;
            auto lookup = [&](int k, int j) {
                const volatile Item* const it = slot(k);
                const int key = j * BN + 32 * (lane >> 3) + 8 * warp + (lane & 7), lp = key / p.ps;
                const int S = it->S, x = key - (S - p.L);
                const bool seen = key < S && (x < 0 || (it->live[x >> 5] >> (x & 31) & 1u));
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
            int k = 0, g = 0, j = 0, last = 0, rows = -1;
            ok = take(0);
            bool more = ok && slot(0)->n > 0;
            if (more) {
                j = slot(0)->j0;
                last = j + slot(0)->n - 1;
                lookup(0, j);
                rows = rows_of();
            }
            // the tile after tile j of piece k: its page ids are requested now
            auto next = [&]() {
                if (j < last) {
                    ++j;
                } else {
                    release(k);
                    ++k;
                    ok = take(k);
                    if (!ok) return;
                    more = slot(k)->n > 0;
                    j = slot(k)->j0;
                    last = j + slot(k)->n - 1;
                }
                if (more) lookup(k, j);
            };
            if constexpr (Q4) {
                // A tile's 4-bit rows are copied to the warp's staging a tile ahead, K when K
                // of the tile before is stored, V likewise, one group of copies each.
                const uint32_t raw_k = base + kOffRaw + warp * 2 * kRawStage, raw_v = raw_k + kRawStage;
                RawTile t;
                if (more) {
                    RawTile::copy(raw_k, p.kc, p.ks, rows, lane);
                    cp_async_commit();
                    RawTile::copy(raw_v, p.vc, p.vs, rows, lane);
                    cp_async_commit();
                }
                while (more) {
                    next();
                    if (!ok) break;
                    const int s = g & 1;
                    cp_async_wait<1>();
                    __syncwarp();
                    t.read(raw_k, lane);
                    if (g >= 2 && !warp_wait(bar(kKEmpty + s), ((g >> 1) - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    t.store<false>(base + kOffK + s * kTile, warp, lane);
                    announce(kKFull + s);
                    if (more) {
                        rows = rows_of();
                        RawTile::copy(raw_k, p.kc, p.ks, rows, lane);
                    }
                    cp_async_commit();
                    cp_async_wait<1>();
                    __syncwarp();
                    t.read(raw_v, lane);
                    if (g >= 2 && !warp_wait(bar(kVEmpty + s), ((g >> 1) - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    if (aborted(abort_flag)) break;
                    t.store<false>(base + kOffV + s * kTile, warp, lane);
                    announce(kVFull + s);
                    ++g;
                    if (more) RawTile::copy(raw_v, p.vc, p.vs, rows, lane);
                    cp_async_commit();
                }
                cp_async_wait<0>();
            } else {
                // K of tile g is requested before V of tile g - 1 is announced, and V of tile
                // g before K of tile g: each has most of a tile's time to arrive.
                while (more) {
                    next();
                    if (!ok) break;
                    const int s = g & 1;
                    if (g >= 2 && !warp_wait(bar(kKEmpty + s), ((g >> 1) - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    if (aborted(abort_flag)) break;
                    copy_tile(base + kOffK + s * kTile, p.kc, rows, warp, lane);
                    cp_async_commit();
                    if (g > 0) {
                        cp_async_wait<1>();
                        announce(kVFull + (s ^ 1));
                    }
                    if (g >= 2 && !warp_wait(bar(kVEmpty + s), ((g >> 1) - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    copy_tile(base + kOffV + s * kTile, p.vc, rows, warp, lane);
                    cp_async_commit();
                    cp_async_wait<1>();
                    announce(kKFull + s);
                    ++g;
                    if (more) rows = rows_of();
                }
                cp_async_wait<0>();
                if (g > 0) announce(kVFull + ((g - 1) & 1));
            }
            if (__any_sync(0xffffffffu, bad_page) && lane == 0) atomicOr(p.flag, PA_FLAG_BAD_PAGE);
        }
        if (!ok && lane == 0) give_up(p, abort_flag);
    } else if (warp < 8) {
        reg_dec<104>();
        if (warp == 4 && lane == 0) {
            // =========================== MMA issuer ===============================
            constexpr uint32_t idS = idesc(Q4, 0, 0);  // Q, K both K-major
            constexpr uint32_t idO = idesc(Q4, 0, 1);  // P K-major, V MN-major
            const uint64_t dQ0 = tc::smem_desc_sw128(base + kOffQ, 16, 1024);
            const uint64_t dK0 = tc::smem_desc_sw128(base + kOffK, 16, 1024);
            const uint64_t dV0 = tc::smem_desc_sw128(base + kOffV, kHalf, 1024);
            auto qk = [&](int t, int buf, int gk) {
                const uint64_t dq = tc::desc_advance(dQ0, buf * kTile), dk = tc::desc_advance(dK0, (gk & 1) * kTile);
                const uint32_t d = tmem + 128u * t;
                tc::mma_bf16_c<0>(d, dq, dk, idS);
#pragma unroll
                for (int kk = 1; kk < kD / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 32;
                    tc::mma_bf16_c<1>(d, tc::desc_advance(dq, off), tc::desc_advance(dk, off), idS);
                }
                tc::commit(bar(kSFull + t));
            };
            auto pv = [&](int t, bool first, int gk) {
                const uint64_t dv = tc::desc_advance(dV0, (gk & 1) * kTile);
                const uint32_t d = tmem + 256u + 128u * t, a = tmem + 128u * t;
                if (first) tc::mma_bf16_ts_c<0>(d, a, dv, idO);
                else tc::mma_bf16_ts_c<1>(d, a, dv, idO);
#pragma unroll
                for (int kk = 1; kk < BN / 16; ++kk)
                    tc::mma_bf16_ts_c<1>(d, a + kk * 8, tc::desc_advance(dv, kk * 16 * 128), idO);
                tc::commit(bar(kODone + t));
            };
            int gk = 0, pc0 = 0, pc1 = 0, oe0 = 0, oe1 = 0;
            bool ok = true;
            for (int k = 0; ok; ++k) {
                ok = mbar_wait(bar(kItemFull + (k & 3)), (k >> 2) & 1);
                if (!ok) break;
                const int nk = slot(k)->n;
                const bool lone = !MULTI || slot(k)->nt == 1;
                mbar_arrive(bar(kItemEmpty + (k & 3)));
                if (nk == 0) break;
                const int jobs = lone ? nk : 2 * nk;
                // job i: key tile, query buffer, and whether it is its key tile's last
                auto tile = [&](int i) { return gk + (lone ? i : i >> 1); };
                auto buf = [&](int i) { return MULTI ? (lone ? 0 : i & 1) : k & 1; };
                auto closes = [&](int i) { return lone || (i & 1); };
                auto issue_qk = [&](int i) {
                    const int x = tile(i);
                    if (!mbar_wait(bar(kKFull + (x & 1)), (x >> 1) & 1)) return false;
                    tc::fence_after_sync();
                    qk(i & 1, buf(i), x);
                    if (closes(i)) tc::commit(bar(kKEmpty + (x & 1)));
                    if (i == jobs - 1) tc::commit(bar(kQEmpty));
                    return true;
                };
                const int qb = MULTI ? 0 : k & 1;
                ok = mbar_wait(bar((Q4 ? kQReady : kQFull) + qb), (MULTI ? k : k >> 1) & 1);
                if (!ok || *abort_flag) break;
                tc::fence_after_sync();
                ok = issue_qk(0) && (jobs < 2 || issue_qk(1));
                for (int i = 0; ok && i < jobs; ++i) {
                    const int t = i & 1, x = tile(i), pc = t ? pc1++ : pc0++, oe = t ? oe1 : oe0;
                    ok = mbar_wait(bar(kVFull + (x & 1)), (x >> 1) & 1) && mbar_wait(bar(kPFull + t), pc & 1);
                    // the previous piece's epilogue has read O
                    if (ok && i < 2 && oe > 0) ok = mbar_wait(bar(kOFree + t), (oe - 1) & 1);
                    if (!ok || *abort_flag) break;
                    tc::fence_after_sync();
                    pv(t, i < 2, x);
                    if (closes(i)) tc::commit(bar(kVEmpty + (x & 1)));
                    if (i + 2 < jobs) ok = issue_qk(i + 2);
                }
                if (!ok || *abort_flag) break;
                gk += nk;
                ++oe0;
                if (jobs > 1) ++oe1;
            }
            if (!ok) give_up(p, abort_flag);
            // nothing of ours may still be running when TMEM is freed
            tc::commit(bar(kMmaDone));
            if (!mbar_wait(bar(kMmaDone), 0)) give_up(p, abort_flag);
        } else if (warp == 7) {
            // ==================== pieces and query tiles =============================
            const uint64_t policy = l2_policy_evict_first();
            const int start = static_cast<int>(blockIdx.x) * share[1], end = min(start + share[1], share[0]);
            int b = 0, S = 0, kvh = 0, mp = 0, ng = 0, seg = end;  // seg: first position of the segment
            if (start < end) {
                b = share[2];
                S = seq_len(p, b);
                ng = key_tiles(S);
                const int i = (start - share[3]) / (kSegCost + ng);
                kvh = i / p.nPairs;
                mp = i - kvh * p.nPairs;
                seg = share[3] + i * (kSegCost + ng);
            }
            int4 crossing = make_int4(-1, 0, 0, 0);
            int before0 = 0, before1 = 0, loads = 0;
            bool ok = true;
            for (int k = 0;; ++k) {
                // this share's key tiles of the segment (none: the share ends before them)
                int j0 = 0, n = 0;
                if (seg < end) {
                    j0 = max(0, start - seg - kSegCost);
                    n = max(0, min(ng, end - seg - kSegCost) - j0);
                }
                if (k >= 4 && !warp_wait(bar(kItemEmpty + (k & 3)), ((k >> 2) - 1) & 1)) {
                    ok = false;
                    break;
                }
                volatile Item* const o = slot(k);
                if (n > 0 && (j0 + n) * BN > S - p.L) {
                    const uint32_t* const m = p.mask + static_cast<long long>(b) * p.L * p.W;
                    if (p.W <= 4) {  // a lane per draft
                        for (int w = 0; w < p.W; ++w) {
                            const int i = 32 * w + lane;
                            uint32_t any = 0u;
                            for (int x = 0; x < p.W; ++x)
                                if (i < p.L) any |= __ldg(m + static_cast<long long>(i) * p.W + x);
                            any = __ballot_sync(0xffffffffu, any != 0u);
                            if (lane == 0) o->live[w] = any;
                        }
                    } else {  // a lane per word
                        for (int w = 0; w < p.W; ++w) {
                            uint32_t bits = 0u;
#pragma unroll 8
                            for (int i = 0; i < 32; ++i) {
                                const int row = 32 * w + i;
                                const uint32_t word = row < p.L && lane < p.W ? __ldg(m + static_cast<long long>(row) * p.W + lane) : 0u;
                                bits |= (__any_sync(0xffffffffu, word != 0u) ? 1u : 0u) << i;
                            }
                            if (lane == 0) o->live[w] = bits;
                        }
                    }
                }
                const int nt = !MULTI || 2 * mp + 1 >= p.nM ? 1 : 2;
                if (lane == 0) {
                    o->b = b;
                    o->S = S;
                    o->kvh = kvh;
                    o->mp = mp;
                    o->ng = ng;
                    o->j0 = j0;
                    o->n = n;
                    o->nt = nt;
                    const int n0 = nt == 1 ? (n + 1) / 2 : n, n1 = nt == 1 ? n / 2 : n;
                    o->jobs[0] = n0;
                    o->jobs[1] = n1;
                    o->before[0] = before0;
                    o->before[1] = before1;
                    before0 += n0;
                    before1 += n1;
                    if (n > 0 && j0 == 0 && n < ng)  // it ends in a later share
                        crossing = make_int4(b, kvh, mp, (seg + kSegCost + ng - 1) / share[1]);
                    mbar_arrive(bar(kItemFull + (k & 3)));
                }
                __syncwarp();
                if (n == 0 || aborted(abort_flag)) break;
                // its query tiles, when the products of the last piece in the buffer are done
                const int ahead = MULTI ? 1 : 2, qb = MULTI ? 0 : k & 1;
                if (k >= ahead && !warp_wait(bar(kQEmpty), (k - ahead) & 1)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    const int row = (b * p.H_kv + kvh) * p.R + 2 * mp * BM;
                    mbar_arrive_expect_tx(bar(kQFull + qb), static_cast<uint32_t>(nt * p.q_box) * 256u);
                    for (int t = 0; t < nt; ++t) {
                        const uint32_t dst = base + kOffQ + (qb + t) * kTile;
                        tc::tma_load_2d(dst, &qmap, 0, row + t * BM, bar(kQFull + qb), policy);
                        tc::tma_load_2d(dst + kHalf, &qmap, 64, row + t * BM, bar(kQFull + qb), policy);
                    }
                }
                ++loads;
                __syncwarp();
                // on to the next segment
                seg += kSegCost + ng;
                if (seg >= end) continue;
                if (++mp == p.nPairs) {
                    mp = 0;
                    if (++kvh == p.H_kv) {
                        kvh = 0;
                        do S = seq_len(p, ++b);
                        while (S == 0);
                        ng = key_tiles(S);
                    }
                }
            }
            if (lane == 0) p.split[blockIdx.x] = crossing;
            // no copy may land after the CTA's shared memory is gone
            for (int x = MULTI ? 1 : 2; x >= 1; --x)
                if (loads >= x) {
                    const int k = loads - x, qb = MULTI ? 0 : k & 1;
                    if (!warp_wait(bar(kQFull + qb), (MULTI ? k : k >> 1) & 1)) ok = false;
                }
            if (!ok && lane == 0) give_up(p, abort_flag);
        }
        __syncwarp();
    } else {
        // ============================== softmax =======================================
        reg_inc<168>();
        const int t = (warp - 8) >> 2, q4 = warp & 3, r = q4 * 32 + lane;  // slot, lane quarter, row
        const uint32_t trow = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
        int xc = 0;  // B's states handed over, two slots in turn
        bool ok = true;
        for (int k = 0;; ++k) {
            ok = take(k);
            if (!ok || slot(k)->n == 0) break;
            const int nk = slot(k)->jobs[t], sc = slot(k)->before[t], S = slot(k)->S, first = S - p.L;
            const bool lone = !MULTI || slot(k)->nt == 1;
            const int m = 2 * slot(k)->mp + (lone ? 0 : t);  // query tile
            const int rows = p.R - m * BM;                    // of which a tile has at most BM
            const bool busy = q4 * 32 < rows, valid = r < rows;
            const int l = (m * BM + r) % p.L;  // draft
            const uint32_t* const mask = p.mask + (static_cast<long long>(slot(k)->b) * p.L + l) * p.W;
            float c = fmaxf(p.scale_log2, FLT_MIN);  // (scale 0: -inf stays -inf)
            if constexpr (Q4) {
                // A's rows (a lone tile) or each tile's own, in place to f16, the largest
                // value in [2^14, 2^15)
                const int buf = MULTI ? (lone ? 0 : t) : k & 1, qb = MULTI ? 0 : k & 1;
                float* const down = reinterpret_cast<float*>(sbase + kOffQScale) + buf * BM + r;
                if (!lone || t == 0) {
                    ok = warp_wait(bar(kQFull + qb), (MULTI ? k : k >> 1) & 1);
                    if (!ok) break;
                    const uint32_t qrow = base + kOffQ + buf * kTile;
                    if (busy) {
                        uint4 v[16];
                        float mx = 0.f;
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(v[c].x), "=r"(v[c].y), "=r"(v[c].z), "=r"(v[c].w)
                                         : "r"(qrow + (c >> 3) * kHalf + sw128(r, c & 7)));
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
                            sts128(qrow + (c >> 3) * kHalf + sw128(r, c & 7), pack_f16x2(f[0].x * up, f[0].y * up),
                                   pack_f16x2(f[1].x * up, f[1].y * up), pack_f16x2(f[2].x * up, f[2].y * up),
                                   pack_f16x2(f[3].x * up, f[3].y * up));
                        }
                        *down = dn;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(kQReady + qb));
                        if (MULTI && lone) mbar_arrive(bar(kQReady + qb));  // for B's warp, which has none
                    }
                }
                // (B, without a job in a piece, must not wait: the pieces can run ahead of it)
                if (nk > 0) {
                    ok = warp_wait(bar(kQReady + qb), (MULTI ? k : k >> 1) & 1);
                    if (!ok) break;
                    if (busy) c = fmaxf(*down * p.scale_log2, FLT_MIN);
                }
            }
            const int tail = first_tail(S);
            float mrow = neg_inf();
            float2 lsum = make_float2(0.f, 0.f);
            for (int j = 0; j < nk; ++j) {
                const int jt = slot(k)->j0 + (lone ? 2 * j + t : j);  // key tile
                uint32_t see[4];
                if (busy && jt >= tail) {  // this row's bits of the tile, while S is on its way
                    const int x = jt * BN - first;
                    const int w0 = x >> 5, sh = x & 31;  // (floor: words before the drafts are all ones)
                    uint32_t w[5];
#pragma unroll
                    for (int i = 0; i < 5; ++i) {
                        const int wi = w0 + i;
                        w[i] = wi < 0 ? 0xffffffffu : wi < p.W ? __ldg(mask + wi) & slot(k)->live[wi] : 0u;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) see[i] = __funnelshift_r(w[i], w[i + 1], sh);
                }
                ok = warp_wait(bar(kSFull + t), (sc + j) & 1);
                if (!ok || aborted(abort_flag)) break;
                if (busy) {
                    tc::fence_after_sync();
                    float x[4][32];
#pragma unroll
                    for (int cc = 0; cc < 4; ++cc) tc::ld32(trow + 128u * t + cc * 32, x[cc]);
                    tc::wait_ld();
                    if (jt >= tail) {
#pragma unroll
                        for (int cc = 0; cc < 4; ++cc)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(see[cc] >> e & 1u)) x[cc][e] = neg_inf();
                    }
                    float mq[4];
#pragma unroll
                    for (int cc = 0; cc < 4; ++cc) {
                        mq[cc] = x[cc][0];
#pragma unroll
                        for (int e = 1; e < 31; e += 2) mq[cc] = fmax3(mq[cc], x[cc][e], x[cc][e + 1]);
                        mq[cc] = fmaxf(mq[cc], x[cc][31]);
                    }
                    const float mt = fmax3(mq[0], mq[1], fmaxf(mq[2], mq[3])) * c;
                    const bool grow = mt > mrow + kLazyRescaleLog2;
                    const bool any_grow = __any_sync(0xffffffffu, grow);
                    const float alpha = grow ? fast_exp2(mrow - mt) : 1.f;  // 2^-inf = 0 at the start
                    if (grow) mrow = mt;
                    const float mu = mrow == neg_inf() ? 0.f : mrow;
                    const float2 c2 = make_float2(c, c), nm2 = make_float2(-mu, -mu);
                    float2 ts = make_float2(0.f, 0.f);
                    uint32_t pw[64];
#pragma unroll
                    for (int i = 0; i < 64; ++i) {
                        const int cc = i >> 4, e = (i & 15) * 2;
                        const float2 y = __ffma2_rn(make_float2(x[cc][e], x[cc][e + 1]), c2, nm2);
                        const float2 ex = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                        pw[i] = Q4 ? pack_f16x2(ex.x, ex.y) : pack_bf16x2(ex.x, ex.y);
                        ts = __fadd2_rn(ts, Q4 ? ex : bf16x2_to_float2(pw[i]));
                    }
                    lsum.x = lsum.x * alpha + ts.x;
                    lsum.y = lsum.y * alpha + ts.y;
                    // O is rescaled once this slot's previous P V is done
                    if (any_grow && j > 0) {
                        ok = warp_wait(bar(kODone + t), (sc + j - 1) & 1);
                        if (!ok || aborted(abort_flag)) break;
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
                    }
                    // P over the first 64 columns of this slot's S (read above)
                    tc::st32(trow + 128u * t, *reinterpret_cast<const uint32_t(*)[32]>(pw));
                    tc::st32(trow + 128u * t + 32, *reinterpret_cast<const uint32_t(*)[32]>(pw + 32));
                    tc::wait_st();
                    tc::fence_before_sync();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kPFull + t));
            }
            if (!ok || aborted(abort_flag)) break;
            const volatile Item* const it = slot(k);
            float l1 = lsum.x + lsum.y;
            if (lone && t == 1) {  // A joins this half with its own
                if (nk > 0) {
                    float2* const x = reinterpret_cast<float2*>(sbase + kOffX) + (xc & 1) * BM + r;
                    *x = make_float2(mrow, l1);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kXFull + (xc & 1)));
                    ++xc;
                }
                release(k);
                continue;
            }
            const bool full = it->n == it->ng;
            // (a full piece has tail tiles)
            const bool drafted = it->live[l >> 5] >> (l & 31) & 1u;
            const long long row = (static_cast<long long>(it->b) * p.H_kv + it->kvh) * p.R + m * BM + r;
            const long long part = ((2ll * blockIdx.x + (it->j0 > 0 ? 0 : 1)) * 2 + (lone ? 0 : t)) * BM + r;
            const int nb = lone ? it->jobs[1] : 0;  // jobs of the other half
            float own = 1.f, other = 0.f;
            if (nb > 0) {
                ok = warp_wait(bar(kXFull + (xc & 1)), (xc >> 1) & 1);
                if (!ok) break;
                const float2 x = reinterpret_cast<const float2*>(sbase + kOffX)[(xc & 1) * BM + r];
                ++xc;
                if (x.y != 0.f) {
                    const float M = fmaxf(mrow, x.x);
                    own = fast_exp2(mrow - M);
                    other = fast_exp2(x.x - M);
                    l1 = l1 * own + x.y * other;
                    mrow = M;
                }
                ok = warp_wait(bar(kODone + 1), (it->before[1] + nb - 1) & 1);
                if (!ok) break;
            }
            if (!full && valid) p.part_ml[part] = make_float2(mrow, l1);
            ok = warp_wait(bar(kODone + t), (sc + nk - 1) & 1);
            if (!ok) break;
            if (busy) {
                tc::fence_after_sync();
                const float inv = l1 == 0.f ? 0.f : 1.f / l1;
#pragma unroll 1
                for (int cc = 0; cc < 4; ++cc) {
                    float o[32];
                    __syncwarp();
                    tc::ld32(trow + 256u + 128u * t + cc * 32, o);
                    tc::wait_ld();
                    if (nb > 0) {  // (uniform)
                        float o2[32];
                        tc::ld32(trow + 256u + 128u + cc * 32, o2);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = o[e] * own + o2[e] * other;
                    }
                    if (!valid) continue;
                    if (full) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = drafted ? pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv) : 0u;
                        uint16_t* const dst = p.out + row * kD + cc * 32;
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
                mbar_arrive(bar(kOFree + t));
                if (nb > 0) mbar_arrive(bar(kOFree + 1));
            }
            release(k);
        }
        if (!ok && lane == 0) give_up(p, abort_flag);
    }

    // ---- tear-down: free TMEM once every role is done ---------------------------
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 4) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

// Merges the partial states of the segments that cross shares: CTA y + ny c takes rows
// 8 y .. of the segment that starts in share c, one a warp, four partial states in flight.
constexpr int kMergeRows = 8;
__global__ void __launch_bounds__(256) tree_merge_kernel(const TileParams p, int ny) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = static_cast<int>(blockIdx.x) / ny, rr = kMergeRows * (static_cast<int>(blockIdx.x) - c * ny) + warp;
    pdl_wait_primary();
    const int4 sp = p.split[c];
    const int in_head = sp.z * 2 * BM + rr;
    if (sp.x < 0 || in_head >= p.R) return;
    const int t = rr >> 7, r = rr & 127, l = in_head % p.L;
    const uint32_t* const m = p.mask + (static_cast<long long>(sp.x) * p.L + l) * p.W;
    const bool drafted = __any_sync(0xffffffffu, lane < p.W && __ldg(m + lane) != 0u);
    float M = neg_inf(), sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = 4;
    for (int k = c; k <= sp.w && drafted; k += U) {
        float2 v[U];
        float4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            v[u] = make_float2(neg_inf(), 0.f);
            if (k + u > sp.w) continue;
            const long long slot = ((2ll * (k + u) + (k + u == c ? 1 : 0)) * 2 + t) * BM + r;
            v[u] = p.part_ml[slot];
            x[u] = *reinterpret_cast<const float4*>(p.part_o + slot * kD + 4 * lane);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (v[u].y == 0.f) continue;  // no key (x was not written)
            const float mx = fmaxf(M, v[u].x), a = fast_exp2(M - mx), b = fast_exp2(v[u].x - mx);
            M = mx;
            sum = sum * a + v[u].y * b;
            acc.x = acc.x * a + x[u].x * b;
            acc.y = acc.y * a + x[u].y * b;
            acc.z = acc.z * a + x[u].z * b;
            acc.w = acc.w * a + x[u].w * b;
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // (0: a row without keys; NaN stays)
    const long long row = (static_cast<long long>(sp.x) * p.H_kv + sp.y) * p.R + in_head;
    *reinterpret_cast<uint2*>(p.out + row * kD + 4 * lane) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

struct TilePlan {
    size_t split_off, ml_off, o_off, total;
};

// (the same for every shape)
TilePlan plan(int sm_count) {
    TilePlan t;
    const size_t slots = 2ull * sm_count * 2 * BM;
    t.split_off = kFlagBytes;
    t.ml_off = align_up(t.split_off + 16ull * sm_count, 256);
    t.o_off = align_up(t.ml_off + slots * 8, 256);
    t.total = t.o_off + slots * kD * 4;
    return t;
}

template <Source SRC, bool MULTI>
pa_status launch_tiles(const TileParams& p, const CUtensorMap* maps, const TreeCall& c) {
    static int attr_done[64] = {0};
    if (!attr_done[c.dev.device]) {
        if (cudaFuncSetAttribute(tree_tile_kernel<SRC, MULTI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 smem_bytes(SRC)) != cudaSuccess)
            return PA_ERR_CUDA;
        attr_done[c.dev.device] = 1;
    }
    tree_tile_kernel<SRC, MULTI><<<static_cast<unsigned>(c.dev.sm_count), kThreads, smem_bytes(SRC), c.stream>>>(
        p, maps[0], maps[1], maps[2]);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
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

bool tree_tiles_supported(const pa_shape& sh) {
    const long long R = static_cast<long long>(sh.H_q / sh.H_kv) * sh.L;
    const long long cap = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    const long long pairs = (R + 2 * BM - 1) / (2 * BM);
    // costs are counted in an int
    return sh.dtype == PA_BF16 && static_cast<long long>(sh.B) * sh.H_kv * pairs * (cap / BN + 1 + kSegCost) < INT_MAX / 2;
}

size_t tree_tiles_workspace_bytes(int sm_count) { return plan(sm_count).total; }

pa_status tree_tiles_launch(const TreeCall& c) {
    const pa_shape& sh = c.sh;
    if (c.dev.smem_optin < smem_bytes(kQ4)) return PA_ERR_UNSUPPORTED;
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
    p.out = static_cast<uint16_t*>(c.out);
    p.flag = reinterpret_cast<uint32_t*>(ws);
    p.part_ml = reinterpret_cast<float2*>(ws + t.ml_off);
    p.part_o = reinterpret_cast<float*>(ws + t.o_off);
    p.split = reinterpret_cast<int4*>(ws + t.split_off);
    p.B = sh.B;
    p.H_kv = sh.H_kv;
    p.R = sh.H_q / sh.H_kv * sh.L;
    p.L = sh.L;
    p.W = tree_words(sh.L);
    p.nM = (p.R + BM - 1) / BM;
    p.nPairs = (p.nM + 1) / 2;
    p.num_pages = sh.num_pages;
    p.ps = sh.page_size;
    p.max_npg = sh.max_pages_per_seq;
    p.pool_rows = sh.num_pages * sh.H_kv * sh.page_size;
    p.box = gcd_int(sh.page_size, BN);
    p.q_box = std::min(BM, (p.R + 7) / 8 * 8);
    p.max_S = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    p.scale_log2 = c.scale * 1.4426950408889634f;
    p.out32 = reinterpret_cast<uintptr_t>(c.out) % 32 == 0;
    const bool tma = !c.ks && sh.page_size % 8 == 0;
    CUtensorMap maps[3];
    if (!make_map(&maps[0], c.q, static_cast<long long>(sh.B) * sh.H_q * sh.L, p.q_box)) return PA_ERR_CUDA;
    maps[1] = maps[2] = maps[0];
    if (tma && (!make_map(&maps[1], c.kc, p.pool_rows, p.box) || !make_map(&maps[2], c.vc, p.pool_rows, p.box)))
        return PA_ERR_CUDA;
    pa_status st;
    if (p.nM > 1)
        st = c.ks  ? launch_tiles<kQ4, true>(p, maps, c)
             : tma ? launch_tiles<kTma, true>(p, maps, c)
                   : launch_tiles<kCopy, true>(p, maps, c);
    else
        st = c.ks  ? launch_tiles<kQ4, false>(p, maps, c)
             : tma ? launch_tiles<kTma, false>(p, maps, c)
                   : launch_tiles<kCopy, false>(p, maps, c);
    if (st != PA_OK) return st;
    const int ny = (std::min(p.R, 2 * BM) + kMergeRows - 1) / kMergeRows;
    return launch_dependent(tree_merge_kernel, dim3(static_cast<unsigned>(c.dev.sm_count * ny)), 256, 0, c.stream, p, ny)
               ? PA_OK
               : PA_ERR_CUDA;
}

}  // namespace pa
