// tiles.cu -- many query rows over 4-bit pages, or over bf16 pages with key weights, on
// tcgen05 tensor cores.
//
// The attention of walk.cu for bf16 queries with many rows per kv head: S = Q K^T
// and O += P V with 128 x 128 tiles, K and V dequantised to f16 on chip (a 4-bit
// value is exact in f16), Q scaled by a power of two per row into f16's range
// (exact), P rounded to f16 (2^-12), max, sums and O in fp32.  Row sums add the
// unrounded weights, so the log-sum-exp that the key weights need is exact.  Over bf16
// pages Q, K, V and P are bf16 (P rounded to 2^-9).
//
// Layout on GB300: one CTA per SM, four warpgroups.
//   * The 128 rows of a query tile are Lt = 128 / G consecutive positions of the
//     G heads that share a kv head; a segment is a pair of tiles A, B of one
//     (sequence, kv head), and its units are the 128-key tiles that its rows see.
//     The units of all segments are cut into equal shares, one per CTA, so ragged
//     contexts leave no SM idle; a segment that crosses shares leaves fp32 partial
//     states that tile_merge_kernel joins.
//   * Warps 0-3 read codes and scales (a tile ahead, in registers), dequantise and
//     store K and V tiles into two-slot rings in shared memory in the 128-byte
//     swizzle the MMA reads, hidden behind the tile's products; bf16 rows come by
//     16-byte asynchronous copies.  No dequantised byte ever leaves the SM.
//   * Warp 4 issues tcgen05.mma in the order PV_A(j), S_A(j+1), PV_B(j), S_B(j+1):
//     one tile's softmax overlaps the other's products.
//   * Warps 8-11 (tile A) and 12-15 (tile B) have one query row per thread: they
//     stage Q, run the softmax from TMEM, put P back into TMEM over S, and write
//     O / l.  The next segment's Q is staged before the epilogue.
//   * Warp 7 publishes the pieces of segments in a ring of four slots.
//   * A last query tile of at most 8 rows is no tensor-core tile: warps 5 and 6
//     take those rows over every staged K/V tile with warp-level MMA.
//   * All waits are bounded; on a timeout the CTA records PA_FLAG_TIMEOUT, frees
//     its TMEM and exits.
//
// Two query tiles are bound by the products as they are issued (about 3600 cycles of a
// key tile's 4200, both operands of Q K^T from shared memory).  One query tile (ONE) would
// wait for its own chain of product, softmax and product: so both softmax warpgroups take
// it, each every other key tile, which leaves the dequantisation as the bound.  Measured
// with the merge (G = 4, H_kv = 8): 8 sequences of 1000 .. 8000 4-bit keys 51 us at 16 or 32
// positions (63 with one warpgroup), 74 at 64, 88 at 65 (a last tile of 4 rows); 64 of
// 500 .. 2000 100, 143, 184.
#include <algorithm>
#include <cfloat>
#include <climits>

#include "cache.h"
#include "ptx.cuh"
#include "stage.cuh"
#include "tc.cuh"

namespace pa {
namespace {

constexpr int kD = kHeadDim;
constexpr int BM = 128, BN = 128;  // query rows and keys of a tile
constexpr int kThreads = 512;
constexpr uint32_t kTmemCols = 512;  // S of tile t at 128 t, O at 256 + 128 t
constexpr float kLazyRescaleLog2 = 8.0f;
// What a segment's query load, first softmax and epilogue cost, in key tiles: the
// shares count it, or CTAs with many short segments would finish last.
constexpr int kSegCost = 3;
constexpr int kHalf = kStageHalf;    // 128 rows x 64 f16 (one swizzled column block)
constexpr int kTile = 2 * kHalf;
constexpr int kOffQ = 0, kOffK = 2 * kTile, kOffV = 4 * kTile, kOffBar = 6 * kTile;
enum Bar {
    kQFull = 0,
    kQEmpty = 1,  // every Q.K^T of a piece is issued and done
    kKFull = 2,    // + slot
    kKEmpty = 4,   // + slot
    kVFull = 6,    // + slot
    kVEmpty = 8,   // + slot
    kSFull = 10,   // + tile
    kPFull = 12,   // + tile
    kODone = 14,   // + tile
    kOFree = 16,   // + tile
    kMmaDone = 18,
    kItemFull = 19,   // + slot: a piece is published
    kItemEmpty = 23,  // + slot: every role is done with it
    kXFull = 27,      // + slot (ONE): B's max and sum
    kNumBars = 30     // (even: what follows stays 16-byte aligned)
};
constexpr int kOffItems = kOffBar + kNumBars * 8;  // four slots
constexpr int kOffTmemSlot = kOffItems + 4 * 64;
constexpr int kOffAbort = kOffTmemSlot + 8;
constexpr int kOffX = kOffAbort + 8;         // ONE: [2][128] max and sum of B's rows
constexpr int kOffRaw = kOffX + 2 * BM * 8;  // ONE: [warp][K, V] 4-bit rows on their way
// With slack to align the base.  Two tiles' loads go through L1, and with more than 196 KB
// of shared memory an SM keeps 28 KB of it instead of 60: 64 sequences of 500 .. 2000 keys,
// 256 rows, 149 us instead of 141.
constexpr int smem_bytes(bool q4, bool one) {
    return (!one ? kOffX : q4 ? kOffRaw + 4 * 2 * kRawStage : kOffRaw) + 1024;
}
static_assert(kOffRaw % 16 == 0, "16-byte copies");

struct TileParams {
    const uint16_t* q;
    const uint8_t *kc, *ks, *vc, *vs;
    const int32_t* bt;
    const int32_t* ctx;
    uint16_t* out;
    float* lse;  // [(b, kvh, row g * L + l)], or null
    uint32_t* flag;
    float2* part_ml;  // [2 per CTA][tile][128]: max, sum
    float* part_o;    // [2 per CTA][tile][128][D]
    int4* split;      // per CTA: the segment that starts in its share and ends in a later one
    float2* rem_ml;   // [(b, kvh) + CTA][warp][8]
    float* rem_o;     // [(b, kvh) + CTA][warp][8][D]
    int* prefix;      // [B] first unit of a sequence, then units per share
    int B, H_q, H_kv, L, G, Lt, nM, nPairs, num_pages, ps, max_npg, causal;
    int nrem, rem_l0;  // rows of the short last tile (0: none), its first position
    long long max_S;
    float scale_log2;
    int min_per;
    int out32;  // the output is 32-byte aligned
};

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ int seq_len(const TileParams& p, int b, bool& bad) {
    const int S = __ldg(p.ctx + b);
    bad = S < 1 || static_cast<long long>(S) > p.max_S || (p.causal && S < p.L);
    return bad ? 0 : S;
}

// Key tiles that positions up to l_last see.
__device__ __forceinline__ int key_tiles(const TileParams& p, int S, int l_last) {
    return (p.causal ? l_last + S - p.L : S - 1) / BN + 1;
}
// First position past query tile m.
__device__ __forceinline__ int tile_end(const TileParams& p, int m) {
    return min((m + 1) * p.Lt, p.nrem > 0 ? p.rem_l0 : p.L);
}
// Units of a segment; the last one also stages what the remainder rows see.
__device__ __forceinline__ int seg_units(const TileParams& p, int S, int mp) {
    const bool last = mp == p.nPairs - 1;
    return key_tiles(p, S, (last ? p.L : tile_end(p, min(2 * mp + 1, p.nM - 1))) - 1);
}
// Cost of a (sequence, kv head): its segments one after the other, each kSegCost and
// then its key tiles.
__device__ __forceinline__ int head_units(const TileParams& p, int S) {
    if (S == 0) return 0;
    if (!p.causal) return p.nPairs * (kSegCost + (S - 1) / BN + 1);
    int n = p.nPairs * kSegCost;
    for (int mp = 0; mp < p.nPairs; ++mp) n += seg_units(p, S, mp);
    return n;
}

// A piece of a segment: key tiles j0 .. j0 + n - 1 of its ng, tile j at cost
// position seg + kSegCost + j of a share that ends at `end`.
struct Piece {
    int b, S, kvh, mp, ng, seg, j0, n;
    // The first piece at or after position pos, in the segment that holds pos.
    __device__ __forceinline__ void cut(const TileParams& p, int pos, int end) {
        ng = seg_units(p, S, mp);
        j0 = max(0, pos - seg - kSegCost);
        n = max(0, min(ng, end - seg - kSegCost) - j0);
    }
    // pos lies in sequence b, whose first position is pref.
    __device__ __forceinline__ void at(const TileParams& p, int pref, int pos, int end) {
        const int per = head_units(p, S);
        kvh = (pos - pref) / per;
        seg = pref + kvh * per;
        for (mp = 0; pos >= seg + kSegCost + seg_units(p, S, mp); ++mp) seg += kSegCost + seg_units(p, S, mp);
        cut(p, pos, end);
    }
    // The next segment's piece; n = 0 past the share.
    __device__ __forceinline__ void advance(const TileParams& p, int end) {
        seg += kSegCost + ng;
        n = 0;
        if (seg + kSegCost >= end) return;
        if (++mp == p.nPairs) {
            mp = 0;
            if (++kvh == p.H_kv) {
                kvh = 0;
                bool bad;
                do S = seq_len(p, ++b, bad);
                while (S == 0);
            }
        }
        cut(p, seg, end);
    }
    // Key tiles of this piece that query tile t takes: the first of them (one query tile
    // for both: A the even ones, B the odd ones).
    template <bool ONE>
    __device__ __forceinline__ int tiles(const TileParams& p, int t) const {
        if constexpr (ONE) return (n + 1 - t) >> 1;
        const int m = 2 * mp + t;
        if (m >= p.nM) return 0;
        return max(0, min(j0 + n, key_tiles(p, S, tile_end(p, m) - 1)) - j0);
    }
};

// A published piece, read from its slot where it is needed (the roles' registers
// are scarce).  Slot k & 3 holds piece k from kItemFull to kItemEmpty.
struct Item {
    int b, S, kvh, mp, ng, j0, n;  // n = 0: no more
    int tiles[2];
    int before_b;  // key tiles of B in earlier pieces
};
static_assert(sizeof(Item) <= 64, "item slot");

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
// Two weights or query values for the products: f16 next to 4-bit rows, bf16 next to bf16 rows.
template <bool Q4>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return Q4 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}

template <int N>
__device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// ONE: all rows of a (sequence, kv head) fit one query tile, which both softmax
// warpgroups take, each every other key tile; A joins the two states at a piece's end.
template <bool Q4, bool ONE>
__global__ void __launch_bounds__(kThreads, 1) tile_kernel(const TileParams p) {
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

    // ---- this CTA's share ------------------------------------------------------
    {
        int mine = 0, v = 0;
        for (int b = tid; b < p.B; b += kThreads) {
            bool bad;
            const int n = p.H_kv * head_units(p, seq_len(p, b, bad));
            if (b == tid) mine = n;
            v += n;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) sums[warp] = v;
        __syncthreads();
        int total = 0;
        for (int w = 0; w < kThreads / 32; ++w) total += sums[w];
        const int per = max((total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x), p.min_per);
        const int u = static_cast<int>(blockIdx.x) * per;
        if (tid == 0) {
            share[0] = total;
            share[1] = per;
            if (blockIdx.x == 0) p.prefix[p.B] = per;
        }
        int carry = 0;
        for (int b0 = 0; b0 < p.B; b0 += kThreads) {
            const int b = b0 + tid;
            int x = mine;
            if (b0 > 0) {
                bool bad;
                x = b < p.B ? p.H_kv * head_units(p, seq_len(p, b, bad)) : 0;
            }
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
            if (b < p.B) {
                if (blockIdx.x == 0) p.prefix[b] = before;
                if (before <= u && u < before + x) {
                    share[2] = b;
                    share[3] = before;
                }
            }
            for (int w = 0; w < kThreads / 32; ++w) carry += sums[w];
        }
        // sequences that break the contract: zero rows
        for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
            bool bad;
            seq_len(p, b, bad);
            if (!bad) continue;
            if (tid == 0) atomicOr(p.flag, PA_FLAG_BAD_CONTEXT);
            const long long rows = static_cast<long long>(p.H_q) * p.L;
            uint4* const o = reinterpret_cast<uint4*>(p.out + b * rows * kD);
            for (long long i = tid; i < rows * (kD / 8); i += kThreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
            if (p.lse)
                for (long long i = tid; i < rows; i += kThreads) p.lse[b * rows + i] = __int_as_float(0x7f800000);
        }
    }
    // ---- set-up ----------------------------------------------------------------
    if (tid == 0) {
        const int readers = p.nrem > 0 ? 3 : 1;  // the MMA's commit, warps 5 and 6
        mbar_init(bar(kQFull), 8);
        mbar_init(bar(kQEmpty), 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(kKFull + s), 4);
            mbar_init(bar(kKEmpty + s), readers);
            mbar_init(bar(kVFull + s), 4);
            mbar_init(bar(kVEmpty + s), readers);
            mbar_init(bar(kSFull + s), 1);
            mbar_init(bar(kPFull + s), 4);
            mbar_init(bar(kODone + s), 1);
            mbar_init(bar(kOFree + s), 4);
        }
        mbar_init(bar(kMmaDone), 1);
        mbar_init(bar(kXFull), 4);
        mbar_init(bar(kXFull + 1), 4);
        for (int s = 0; s < 4; ++s) {
            mbar_init(bar(kItemFull + s), 1);
            // producers, the MMA thread, softmax warps, warps 5 and 6
            mbar_init(bar(kItemEmpty + s), 4 + 1 + 8 + (p.nrem > 0 ? 2 : 0));
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 4) {
        tc::tmem_alloc(base + kOffTmemSlot, kTmemCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    auto slot = [&](int k) { return reinterpret_cast<volatile Item*>(sbase + kOffItems + 64 * (k & 3)); };
    auto take = [&](int k) { return warp_wait(bar(kItemFull + (k & 3)), (k >> 2) & 1); };  // a whole warp
    auto release = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kItemEmpty + (k & 3)));
    };

    if (warp < 4) {
        // ========================= K/V producers ==================================
        reg_dec<72>();
        // pool rows of the next tile, lane 8 i + r: key 32 i + 8 warp + r
        int page = 0, in_page = -1, row_base = 0;  // in_page: the key's slot, -1 past the context
        bool bad_page = false;
        auto lookup = [&](int b, int S, int kvh, int j) {
            const int key = j * BN + 32 * (lane >> 3) + 8 * warp + (lane & 7);
            const int lp = key / p.ps;
            in_page = key < S ? key - lp * p.ps : -1;
            page = key < S ? __ldg(p.bt + static_cast<long long>(b) * p.max_npg + lp) : 0;
            row_base = kvh;
        };
        auto rows_of = [&]() {
            const bool ok = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages);
            bad_page |= in_page >= 0 && !ok;
            return in_page >= 0 && ok ? (page * p.H_kv + row_base) * p.ps + in_page : -1;
        };
        bool ok = take(0);
        int k = 0, g = 0;  // piece, tiles so far
        if constexpr (Q4 && !ONE) if (ok && slot(0)->n > 0) {
            RawTile rk, rv;
            int j = slot(0)->j0, last = j + slot(0)->n - 1;
            lookup(slot(0)->b, slot(0)->S, slot(0)->kvh, j);
            int rows = rows_of();
            rk.request(p.kc, p.ks, rows, lane);
            rv.request(p.vc, p.vs, rows, lane);
            for (bool more = true; more;) {  // tile j of piece k is in registers
                // the tile after it: its page ids are requested now
                if (j < last) {
                    ++j;
                } else {
                    release(k);
                    ++k;
                    ok = take(k);
                    if (!ok) break;
                    more = slot(k)->n > 0;
                    j = slot(k)->j0;
                    last = j + slot(k)->n - 1;
                }
                if (more) lookup(slot(k)->b, slot(k)->S, slot(k)->kvh, j);
                const int s = g & 1;
                if (g >= 2 && !warp_wait(bar(kKEmpty + s), ((g >> 1) - 1) & 1)) {
                    ok = false;
                    break;
                }
                rk.store<false>(base + kOffK + s * kTile, warp, lane);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kKFull + s));
                if (more) {
                    rows = rows_of();
                    rk.request(p.kc, p.ks, rows, lane);
                }
                if (g >= 2 && !warp_wait(bar(kVEmpty + s), ((g >> 1) - 1) & 1)) {
                    ok = false;
                    break;
                }
                if (aborted(abort_flag)) break;
                rv.store<false>(base + kOffV + s * kTile, warp, lane);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kVFull + s));
                ++g;
                if (more) rv.request(p.vc, p.vs, rows, lane);
            }
        }
        // One query tile: a key tile's time is short, and the loads above, whose wait comes
        // right after their issue (1500 cycles a tile), would set it.  The rows are copied to this warp's staging
        // a tile ahead: K of tile g + 1 when K of tile g is stored, V likewise, one group of
        // copies each.  (64 rows over 8 sequences of 1000 .. 8000 keys: loads 61 us, copies
        // 59, copies and both warpgroups on the tile 52.  Two tiles of 260 rows: 88, 90.)
        if constexpr (Q4 && ONE) if (ok && slot(0)->n > 0) {
            const uint32_t raw_k = base + kOffRaw + warp * 2 * kRawStage, raw_v = raw_k + kRawStage;
            RawTile raw;
            int j = slot(0)->j0, last = j + slot(0)->n - 1;
            lookup(slot(0)->b, slot(0)->S, slot(0)->kvh, j);
            int rows = rows_of();
            RawTile::copy(raw_k, p.kc, p.ks, rows, lane);
            cp_async_commit();
            RawTile::copy(raw_v, p.vc, p.vs, rows, lane);
            cp_async_commit();
            for (bool more = true; more;) {  // tile j of piece k is on its way
                // the tile after it: its page ids are requested now
                if (j < last) {
                    ++j;
                } else {
                    release(k);
                    ++k;
                    ok = take(k);
                    if (!ok) break;
                    more = slot(k)->n > 0;
                    j = slot(k)->j0;
                    last = j + slot(k)->n - 1;
                }
                if (more) lookup(slot(k)->b, slot(k)->S, slot(k)->kvh, j);
                const int s = g & 1;
                cp_async_wait<1>();
                __syncwarp();
                raw.read(raw_k, lane);
                if (g >= 2 && !warp_wait(bar(kKEmpty + s), ((g >> 1) - 1) & 1)) {
                    ok = false;
                    break;
                }
                raw.store<false>(base + kOffK + s * kTile, warp, lane);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kKFull + s));
                if (more) {
                    rows = rows_of();
                    RawTile::copy(raw_k, p.kc, p.ks, rows, lane);
                }
                cp_async_commit();
                cp_async_wait<1>();
                __syncwarp();
                raw.read(raw_v, lane);
                if (g >= 2 && !warp_wait(bar(kVEmpty + s), ((g >> 1) - 1) & 1)) {
                    ok = false;
                    break;
                }
                if (aborted(abort_flag)) break;
                raw.store<false>(base + kOffV + s * kTile, warp, lane);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kVFull + s));
                ++g;
                if (more) RawTile::copy(raw_v, p.vc, p.vs, rows, lane);
                cp_async_commit();
            }
            cp_async_wait<0>();
        }
        if constexpr (!Q4) {
            // K of tile g is requested before V of tile g - 1 is announced, and V of tile
            // g before K of tile g: each has most of a tile's time to arrive.
            auto announce = [&](int b) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(b));
            };
            int j = 0, last = 0, rows = -1;
            bool more = ok && slot(0)->n > 0;
            if (more) {
                j = slot(0)->j0;
                last = j + slot(0)->n - 1;
                lookup(slot(0)->b, slot(0)->S, slot(0)->kvh, j);
                rows = rows_of();
            }
            while (more) {
                if (j < last) {
                    ++j;
                } else {
                    release(k);
                    ++k;
                    ok = take(k);
                    if (!ok) break;
                    more = slot(k)->n > 0;
                    j = slot(k)->j0;
                    last = j + slot(k)->n - 1;
                }
                if (more) lookup(slot(k)->b, slot(k)->S, slot(k)->kvh, j);
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
        if (!ok && lane == 0) give_up(p, abort_flag);
        if (__any_sync(0xffffffffu, bad_page) && lane == 0) atomicOr(p.flag, PA_FLAG_BAD_PAGE);
    } else if (warp < 8) {
        reg_dec<104>();
        if (warp == 4 && lane == 0) {
            // =========================== MMA issuer ===============================
            constexpr uint32_t idS = idesc(Q4, 0, 0);  // Q, K both K-major
            constexpr uint32_t idO = idesc(Q4, 0, 1);  // P K-major, V MN-major
            const uint64_t dQ[2] = {tc::smem_desc_sw128(base + kOffQ, 16, 1024),
                                    tc::smem_desc_sw128(base + kOffQ + kTile, 16, 1024)};
            const uint64_t dK0 = tc::smem_desc_sw128(base + kOffK, 16, 1024);
            const uint64_t dV0 = tc::smem_desc_sw128(base + kOffV, kHalf, 1024);
            auto qk = [&](int t, int gk) {
                const uint64_t dq = t ? dQ[1] : dQ[0], dk = tc::desc_advance(dK0, (gk & 1) * kTile);
                const uint32_t d = tmem + 128u * t;
                tc::mma_bf16_c<0>(d, dq, dk, idS);
#pragma unroll
                for (int kk = 1; kk < kD / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 32;
                    tc::mma_bf16_c<1>(d, tc::desc_advance(dq, off), tc::desc_advance(dk, off), idS);
                }
                tc::commit(bar(kSFull + t));
            };
            auto pv = [&](int t, bool first_tile, int gk) {
                const uint64_t dv = tc::desc_advance(dV0, (gk & 1) * kTile);
                const uint32_t d = tmem + 256u + 128u * t, a = tmem + 128u * t;
                if (first_tile) tc::mma_bf16_ts_c<0>(d, a, dv, idO);
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
                const int n0 = slot(k)->tiles[0], n1 = slot(k)->tiles[1], nk = slot(k)->n;
                mbar_arrive(bar(kItemEmpty + (k & 3)));
                if (nk == 0) break;
                ok = mbar_wait(bar(kQFull), k & 1) && mbar_wait(bar(kKFull + (gk & 1)), (gk >> 1) & 1);
                if (!ok || *abort_flag) break;
                tc::fence_after_sync();
                if constexpr (ONE) {  // key tile j belongs to t = j & 1
                    qk(0, gk);
                    tc::commit(bar(kKEmpty + (gk & 1)));
                    if (nk > 1) {
                        ok = mbar_wait(bar(kKFull + ((gk + 1) & 1)), ((gk + 1) >> 1) & 1);
                        if (!ok || *abort_flag) break;
                        tc::fence_after_sync();
                        qk(1, gk + 1);
                        tc::commit(bar(kKEmpty + ((gk + 1) & 1)));
                    }
                    if (nk <= 2) tc::commit(bar(kQEmpty));
                    for (int j = 0; j < nk; ++j, ++gk) {
                        const int t = j & 1, pc = t ? pc1++ : pc0++, oe = t ? oe1 : oe0;
                        ok = mbar_wait(bar(kVFull + (gk & 1)), (gk >> 1) & 1) && mbar_wait(bar(kPFull + t), pc & 1);
                        // the previous piece's epilogue has read O
                        if (ok && j < 2 && oe > 0) ok = mbar_wait(bar(kOFree + t), (oe - 1) & 1);
                        if (!ok || *abort_flag) break;
                        tc::fence_after_sync();
                        pv(t, j < 2, gk);
                        tc::commit(bar(kVEmpty + (gk & 1)));
                        if (j + 2 < nk) {
                            ok = mbar_wait(bar(kKFull + (gk & 1)), ((gk + 2) >> 1) & 1);
                            if (!ok || *abort_flag) break;
                            tc::fence_after_sync();
                            qk(t, gk + 2);
                            tc::commit(bar(kKEmpty + (gk & 1)));
                            if (j + 3 == nk) tc::commit(bar(kQEmpty));  // the piece's last Q.K^T
                        }
                    }
                    if (!ok || *abort_flag) break;
                    ++oe0;
                    if (n1 > 0) ++oe1;
                    continue;
                }
                if (n0 > 0) qk(0, gk);
                if (n1 > 0) qk(1, gk);
                tc::commit(bar(kKEmpty + (gk & 1)));
                if (nk == 1) tc::commit(bar(kQEmpty));
                for (int j = 0; j < nk; ++j, ++gk) {
                    ok = mbar_wait(bar(kVFull + (gk & 1)), (gk >> 1) & 1);
                    if (!ok || *abort_flag) break;
                    const bool more = j + 1 < nk;
                    if (j < n0) {
                        ok = mbar_wait(bar(kPFull), pc0 & 1);
                        // the previous piece's epilogue has read O
                        if (ok && j == 0 && oe0 > 0) ok = mbar_wait(bar(kOFree), (oe0 - 1) & 1);
                        if (!ok || *abort_flag) break;
                        ++pc0;
                        tc::fence_after_sync();
                        pv(0, j == 0, gk);
                    }
                    if (more) {
                        ok = mbar_wait(bar(kKFull + ((gk + 1) & 1)), ((gk + 1) >> 1) & 1);
                        if (!ok || *abort_flag) break;
                        tc::fence_after_sync();
                        if (j + 1 < n0) qk(0, gk + 1);
                    }
                    if (j < n1) {
                        ok = mbar_wait(bar(kPFull + 1), pc1 & 1);
                        if (ok && j == 0 && oe1 > 0) ok = mbar_wait(bar(kOFree + 1), (oe1 - 1) & 1);
                        if (!ok || *abort_flag) break;
                        ++pc1;
                        tc::fence_after_sync();
                        pv(1, j == 0, gk);
                    }
                    tc::commit(bar(kVEmpty + (gk & 1)));
                    if (more) {
                        if (j + 1 < n1) qk(1, gk + 1);
                        tc::commit(bar(kKEmpty + ((gk + 1) & 1)));
                        if (j + 2 == nk) tc::commit(bar(kQEmpty));  // the piece's last Q.K^T
                    }
                }
                if (!ok || *abort_flag) break;
                if (n0 > 0) ++oe0;
                if (n1 > 0) ++oe1;
            }
            if (!ok) give_up(p, abort_flag);
            // nothing of ours may still be running when TMEM is freed
            tc::commit(bar(kMmaDone));
            if (!mbar_wait(bar(kMmaDone), 0)) give_up(p, abort_flag);
        } else if ((warp == 5 || warp == 6) && p.nrem > 0) {
            // ======================= remainder rows ================================
            // S^T = K Q^T and O^T += V^T P^T (16 keys x 8 rows): lane 4g + t holds
            // keys g and g + 8 of rows 2t and 2t + 1.
            const int wr = warp - 5, g = lane >> 2, t4 = lane & 3;  // keys 64 wr .. of every tile
            const int Lrem = p.L - p.rem_l0;
            int gk = 0;
            bool ok = true;
            for (int k = 0; ok; ++k) {
                ok = take(k);
                if (!ok) break;
                const int n = slot(k)->n, j0 = slot(k)->j0, b = slot(k)->b, kvh = slot(k)->kvh, S = slot(k)->S;
                const bool rem = slot(k)->mp == p.nPairs - 1;
                release(k);
                if (n == 0) break;
                uint32_t qf[8][2];
                float o[8][4], m_r[2] = {neg_inf(), neg_inf()}, l_r[2] = {0.f, 0.f}, qs[2] = {1.f, 1.f};
                int lim[2] = {-1, -1};
                if (rem) {
                    // row g of the remainder: its dims 16 ks + 2t, + 8
                    const int gq = g / Lrem, lq = p.rem_l0 + (g - gq * Lrem);
                    const uint16_t* const row =
                        p.q + ((static_cast<long long>(b) * p.H_q + kvh * p.G + gq) * p.L + lq) * kD;
                    float mx = 0.f;
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        uint32_t w = 0u;
                        if (g < p.nrem) w = __ldg(reinterpret_cast<const uint32_t*>(row + 16 * (k >> 1) + 8 * (k & 1) + 2 * t4));
                        qf[k >> 1][k & 1] = w;
                        const float2 f = bf16x2_to_float2(w);
                        mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    float up, down;
                    f16_scale(mx, up, down);
                    if constexpr (Q4) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float2 f = bf16x2_to_float2(qf[k >> 1][k & 1]);
                            qf[k >> 1][k & 1] = pack_f16x2(f.x * up, f.y * up);
                        }
                    } else {
                        down = 1.f;
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        qs[e] = fmaxf(__shfl_sync(0xffffffffu, down, 8 * t4 + 4 * e) * p.scale_log2, FLT_MIN);
                        const int rr = 2 * t4 + e;
                        if (rr < p.nrem) lim[e] = p.causal ? p.rem_l0 + rr % Lrem + S - p.L : S - 1;
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
                }
                for (int jj = 0; jj < n; ++jj, ++gk) {
                    const int s = gk & 1, key0 = (j0 + jj) * BN + 64 * wr;
                    const uint32_t kb = base + kOffK + s * kTile, vb = base + kOffV + s * kTile;
                    ok = warp_wait(bar(kKFull + s), (gk >> 1) & 1);
                    if (!ok || aborted(abort_flag)) {
                        ok = false;
                        break;
                    }
                    float x[4][4];
                    if (rem) {  // 64 keys as 4 groups of 16: four chains in flight
                        const int r0 = 64 * wr + (lane & 7) + ((lane >> 3) & 1) * 8;
                        // (the next step's fragments are requested before this one's products)
                        uint32_t a[2][4][4];
                        auto load = [&](int ks) {
                            const int c = ks * 2 + (lane >> 4);
#pragma unroll
                            for (int grp = 0; grp < 4; ++grp)
                                ldmatrix_x4(a[ks & 1][grp], kb + (c >> 3) * kHalf + sw128(r0 + 16 * grp, c & 7));
                        };
                        load(0);
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks) {
                            if (ks < 7) load(ks + 1);
#pragma unroll
                            for (int grp = 0; grp < 4; ++grp) {
                                if (ks == 0) mma_first<Q4>(x[grp], a[0][grp], qf[0][0], qf[0][1]);
                                else mma<Q4>(x[grp], a[ks & 1][grp], qf[ks][0], qf[ks][1]);
                            }
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kKEmpty + s));
                    ok = warp_wait(bar(kVFull + s), (gk >> 1) & 1);
                    if (!ok || aborted(abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (rem) {
                        float mt[2] = {neg_inf(), neg_inf()};
#pragma unroll
                        for (int grp = 0; grp < 4; ++grp)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int key = key0 + 16 * grp + g + (e >> 1) * 8;
                                x[grp][e] = key <= lim[e & 1] ? x[grp][e] * qs[e & 1] : neg_inf();
                                mt[e & 1] = fmaxf(mt[e & 1], x[grp][e]);
                            }
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) {
                            mt[0] = fmaxf(mt[0], __shfl_xor_sync(0xffffffffu, mt[0], d));
                            mt[1] = fmaxf(mt[1], __shfl_xor_sync(0xffffffffu, mt[1], d));
                        }
                        const bool g0 = mt[0] > m_r[0] + kLazyRescaleLog2, g1 = mt[1] > m_r[1] + kLazyRescaleLog2;
                        if (__any_sync(0xffffffffu, g0 || g1)) {
                            const float a0 = g0 ? fast_exp2(m_r[0] - mt[0]) : 1.f;
                            const float a1 = g1 ? fast_exp2(m_r[1] - mt[1]) : 1.f;
                            if (g0) m_r[0] = mt[0];
                            if (g1) m_r[1] = mt[1];
                            l_r[0] *= a0;
                            l_r[1] *= a1;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                o[i][0] *= a0;
                                o[i][1] *= a1;
                                o[i][2] *= a0;
                                o[i][3] *= a1;
                            }
                        }
                        const float mu0 = m_r[0] == neg_inf() ? 0.f : m_r[0], mu1 = m_r[1] == neg_inf() ? 0.f : m_r[1];
                        uint32_t pb[4][2];
#pragma unroll
                        for (int grp = 0; grp < 4; ++grp)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const float p0 = fast_exp2(x[grp][2 * h] - mu0), p1 = fast_exp2(x[grp][2 * h + 1] - mu1);
                                l_r[0] += p0;
                                l_r[1] += p1;
                                pb[grp][h] = movmatrix_trans(pack2<Q4>(p0, p1));
                            }
                        // step n: dims 64 (n & 1) .. of group n >> 1
                        const int r = 64 * wr + (lane & 7) + (lane >> 4) * 8;
                        uint32_t a[2][4][4];
                        auto load = [&](int n) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                ldmatrix_x4_trans(a[n & 1][i], vb + (n & 1) * kHalf +
                                                                   sw128(r + 16 * (n >> 1), i * 2 + ((lane >> 3) & 1)));
                        };
                        load(0);
#pragma unroll
                        for (int n = 0; n < 8; ++n) {
                            if (n < 7) load(n + 1);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mma<Q4>(o[4 * (n & 1) + i], a[n & 1][i], pb[n >> 1][0], pb[n >> 1][1]);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kVEmpty + s));
                }
                if (!ok) break;
                if (rem) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        l_r[0] += __shfl_xor_sync(0xffffffffu, l_r[0], d);
                        l_r[1] += __shfl_xor_sync(0xffffffffu, l_r[1], d);
                    }
                    const long long slot = (static_cast<long long>(b) * p.H_kv + kvh + blockIdx.x) * 2 + wr;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int rr = 2 * t4 + e;
                        if (g == 0) p.rem_ml[slot * 8 + rr] = make_float2(m_r[e], l_r[e]);
                        float* const po = p.rem_o + (slot * 8 + rr) * kD;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            po[16 * i + g] = o[i][e];
                            po[16 * i + g + 8] = o[i][2 + e];
                        }
                    }
                }
            }
            if (!ok && lane == 0) give_up(p, abort_flag);
        } else if (warp == 7) {
            // ========================= scheduler ===================================
            Piece it = {};
            const int pos = static_cast<int>(blockIdx.x) * share[1], end = min(pos + share[1], share[0]);
            if (pos < end) {
                bool bad;
                it.b = share[2];
                it.S = seq_len(p, it.b, bad);
                it.at(p, share[3], pos, end);
                if (it.n == 0) it.advance(p, end);  // the share's first segment ends before its first tile here
            }
            int4 crossing = make_int4(-1, 0, 0, 0);
            int before_b = 0;
            for (int k = 0;; ++k) {
                if (k >= 4 && !warp_wait(bar(kItemEmpty + (k & 3)), ((k >> 2) - 1) & 1)) {
                    if (lane == 0) give_up(p, abort_flag);
                    break;
                }
                const int n = it.n;
                if (lane == 0) {
                    volatile Item* const o = slot(k);
                    o->b = it.b;
                    o->S = it.S;
                    o->kvh = it.kvh;
                    o->mp = it.mp;
                    o->ng = it.ng;
                    o->j0 = it.j0;
                    o->n = n;
                    for (int t = 0; t < 2; ++t) o->tiles[t] = n > 0 ? it.template tiles<ONE>(p, t) : 0;
                    o->before_b = before_b;
                    before_b += o->tiles[1];
                    if (n > 0 && it.j0 == 0 && n < it.ng)  // it ends in a later share
                        crossing = make_int4(it.b, it.kvh, it.mp, (it.seg + kSegCost + it.ng - 1) / share[1]);
                    mbar_arrive(bar(kItemFull + (k & 3)));
                }
                __syncwarp();
                if (n == 0 || aborted(abort_flag)) break;
                it.advance(p, end);
            }
            if (lane == 0) p.split[blockIdx.x] = crossing;
        }
        __syncwarp();
    } else {
        // ============================== softmax =======================================
        reg_inc<168>();
        const int t = (warp - 8) >> 2, q4 = warp & 3, r = q4 * 32 + lane;  // tile, lane quarter, row
        const uint32_t trow = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
        const uint32_t qrow = base + kOffQ + t * kTile;
        const int g = r / p.Lt, dl = r - g * p.Lt;
        int sc = 0;  // S fills and P.V products of this tile in earlier pieces
        // ONE: B's states that A has taken, two slots in turn.  Only a piece in which B has
        // key tiles hands one over: B then waited for an S of this piece, hence (kQFull) for
        // every warp of A to be through with the piece before the last one, so a slot is free
        // again when its turn comes.  A piece of one key tile would let B run ahead of A.
        int xc = 0;
        float qs = 1.f;
        bool ok = true;
        // The query rows of piece k, as they are, on their way into this tile's
        // buffer: the warp's 32 rows two at a time, 16 lanes a row.  The tile's last
        // S of the piece before must be done (no one else reads the buffer).
        auto fetch = [&](int k) {
            const int m = 2 * slot(k)->mp + (ONE ? 0 : t), l_end = m < p.nM ? tile_end(p, m) : 0;
            const uint16_t* const head = p.q + (static_cast<long long>(slot(k)->b) * p.H_q + slot(k)->kvh * p.G) * p.L * kD;
            const int c = lane & 15;
            int rr = q4 * 32 + (lane >> 4), gr = rr / p.Lt, dr = rr - gr * p.Lt;
#pragma unroll 4
            for (int i = 0; i < 16; ++i, rr += 2) {
                const int l = m * p.Lt + dr;
                const bool in = gr < p.G && l < l_end;
                const uint16_t* const src = head + (in ? (static_cast<long long>(gr) * p.L + l) * kD + 8 * c : 0);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 qrow + (c >> 3) * kHalf + sw128(rr, c & 7)),
                             "l"(src), "r"(in ? 16 : 0)
                             : "memory");
                for (dr += 2; dr >= p.Lt; dr -= p.Lt) ++gr;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // Each thread's row in place to f16, the largest value in [2^14, 2^15) (bf16 pages:
        // as it is).  The
        // tile of a pair that has nothing to do in a piece must not run ahead: piece k
        // is announced once the products of piece k - 1 are through.
        auto convert = [&](int k) {
            if (k > 0 && !warp_wait(bar(kQEmpty), (k - 1) & 1)) return false;
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncwarp();
            float down = 1.f;
            if constexpr (Q4) {
                uint4 v[16];
                float mx = 0.f;
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(v[c].x), "=r"(v[c].y), "=r"(v[c].z), "=r"(v[c].w)
                                 : "r"(qrow + (c >> 3) * kHalf + sw128(r, c & 7)));
                    const float2 f[4] = {bf16x2_to_float2(v[c].x), bf16x2_to_float2(v[c].y), bf16x2_to_float2(v[c].z),
                                         bf16x2_to_float2(v[c].w)};
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx = fmax3(mx, fabsf(f[e].x), fabsf(f[e].y));
                }
                float up;
                f16_scale(mx, up, down);
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const float2 f[4] = {bf16x2_to_float2(v[c].x), bf16x2_to_float2(v[c].y), bf16x2_to_float2(v[c].z),
                                         bf16x2_to_float2(v[c].w)};
                    sts128(qrow + (c >> 3) * kHalf + sw128(r, c & 7), pack_f16x2(f[0].x * up, f[0].y * up),
                           pack_f16x2(f[1].x * up, f[1].y * up), pack_f16x2(f[2].x * up, f[2].y * up),
                           pack_f16x2(f[3].x * up, f[3].y * up));
                }
            }
            qs = fmaxf(down * p.scale_log2, FLT_MIN);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kQFull));
            return true;
        };
        ok = take(0);
        if (ok && slot(0)->n > 0) {
            fetch(0);
            ok = convert(0);
        }
        for (int k = 0; ok && slot(k)->n > 0; ++k) {
            const int nk = slot(k)->tiles[t];
            int key0 = (slot(k)->j0 + (ONE ? t : 0)) * BN;
            int lim = slot(k)->S - 1, lim_min = lim;  // the last key this row sees, the tile's first
            if (p.causal) {
                const int l0 = (2 * slot(k)->mp + (ONE ? 0 : t)) * p.Lt + slot(k)->S - p.L;
                lim = l0 + dl;
                lim_min = l0;
            }
            bool fetched = false;  // the next piece's query
            const float c = qs;
            float mrow = neg_inf();
            float2 lsum = make_float2(0.f, 0.f);
            for (int j = 0; j < nk; ++j) {
                ok = warp_wait(bar(kSFull + t), (sc + j) & 1);
                if (!ok || aborted(abort_flag)) break;
                tc::fence_after_sync();
                float x[4][32];
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) tc::ld32(trow + 128u * t + cc * 32, x[cc]);
                tc::wait_ld();
                if (j + 1 == nk && __all_sync(0xffffffffu, mbar_try_wait(bar(kItemFull + ((k + 1) & 3)), ((k + 1) >> 2) & 1)) &&
                    slot(k + 1)->n > 0) {
                    fetch(k + 1);
                    fetched = true;
                }
                if (key0 + BN - 1 > lim_min) {
                    const int cmax = lim - key0;
#pragma unroll
                    for (int cc = 0; cc < 4; ++cc)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (cc * 32 + e > cmax) x[cc][e] = neg_inf();
                }
                key0 += ONE ? 2 * BN : BN;
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
                for (int k = 0; k < 64; ++k) {
                    const int cc = k >> 4, e = (k & 15) * 2;
                    const float2 y = __ffma2_rn(make_float2(x[cc][e], x[cc][e + 1]), c2, nm2);
                    const float2 ex = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                    ts = __fadd2_rn(ts, ex);
                    pw[k] = pack2<Q4>(ex.x, ex.y);
                }
                lsum.x = lsum.x * alpha + ts.x;
                lsum.y = lsum.y * alpha + ts.y;
                // O is rescaled once this tile's previous P.V is done
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
                // P over the first 64 columns of this tile's S (read above)
                tc::st32(trow + 128u * t, *reinterpret_cast<const uint32_t(*)[32]>(pw));
                tc::st32(trow + 128u * t + 32, *reinterpret_cast<const uint32_t(*)[32]>(pw + 32));
                tc::wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kPFull + t));
            }
            if (!ok || aborted(abort_flag)) break;
            // the next piece's query, while the last P.V runs
            ok = take(k + 1);
            if (!ok) break;
            if (slot(k + 1)->n > 0) {
                if (!fetched) fetch(k + 1);
                ok = convert(k + 1);
                if (!ok) break;
            }
            const volatile Item* const done = slot(k);
            float l1 = lsum.x + lsum.y;
            if (ONE && t == 1) {  // A joins this half with its own
                if (nk > 0) {
                    float2* const x = reinterpret_cast<float2*>(sbase + kOffX) + (xc & 1) * BM + r;
                    *x = make_float2(mrow, l1);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kXFull + (xc & 1)));
                    ++xc;
                }
                sc += nk;
                release(k);
                continue;
            }
            const int m = 2 * done->mp + t, l = m * p.Lt + dl;
            const bool valid = m < p.nM && g < p.G && l < tile_end(p, m);
            const bool full = done->n == done->ng;
            const long long row = (static_cast<long long>(done->b) * p.H_q + done->kvh * p.G + g) * p.L + l;
            const long long part = ((2ll * blockIdx.x + (done->j0 > 0 ? 0 : 1)) * 2 + t) * BM + r;
            const int nb = ONE ? done->tiles[1] : 0;  // key tiles of the other half
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
                ok = warp_wait(bar(kODone + 1), (done->before_b + nb - 1) & 1);
                if (!ok) break;
            }
            if (!full) p.part_ml[part] = make_float2(mrow, l1);
            if (nk > 0) {
                ok = warp_wait(bar(kODone + t), (sc + nk - 1) & 1);
                if (!ok) break;
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
                        for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
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
                // O of this tile is read: the next piece's first P.V may overwrite it
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(kOFree + t));
                    if (nb > 0) mbar_arrive(bar(kOFree + 1));
                }
            }
            if (full && valid && p.lse) p.lse[row] = l1 == 0.f ? __int_as_float(0x7f800000) : mrow + log2f(l1);
            sc += nk;
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

__device__ __forceinline__ void store_row(const TileParams& p, long long row, int lane, float4 acc, float l, float M) {
    const float inv = l == 0.f ? 0.f : 1.f / l;  // (0: a row without keys; NaN stays)
    *reinterpret_cast<uint2*>(p.out + row * kD + 4 * lane) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lane == 0 && p.lse) p.lse[row] = l == 0.f ? __int_as_float(0x7f800000) : M + log2f(l);
}

// A merged state of one row, four dims a lane.
struct RowState {
    float M, l;
    float4 acc;
    __device__ __forceinline__ void init() {
        M = neg_inf();
        l = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ __forceinline__ void add(const float2 v, const float4 x) {
        if (v.y == 0.f) return;  // no key (x was not written)
        const float m = fmaxf(M, v.x), a = fast_exp2(M - m), b = fast_exp2(v.x - m);
        M = m;
        l = l * a + v.y * b;
        acc.x = acc.x * a + x.x * b;
        acc.y = acc.y * a + x.y * b;
        acc.z = acc.z * a + x.z * b;
        acc.w = acc.w * a + x.w * b;
    }
};

// Rows per merge CTA, one a warp (8, 4 rows, us for the call: 2 sequences of 900 keys, 256
// rows 33, 37; one of 16000 45, 47).
constexpr int kMergeRows = 8;

// Merges the partial states of the segments that cross shares: CTA y + ny c takes rows
// 8 y .. of the segment that starts in share c, four partial states a warp in flight;
// then a CTA for the remainder rows of each (sequence, kv head).
__global__ void __launch_bounds__(256) tile_merge_kernel(const TileParams p, int shares, int ny) {
    pdl_launch_dependents();
    pdl_wait_primary();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    RowState st;
    st.init();
    const int rest = static_cast<int>(blockIdx.x) - shares * ny;
    if (rest < 0) {
        const int c = static_cast<int>(blockIdx.x) / ny, rr = kMergeRows * (static_cast<int>(blockIdx.x) - c * ny) + warp;
        const int4 sp = p.split[c];
        if (sp.x < 0) return;
        const int t = rr >> 7, r = rr & 127, m = 2 * sp.z + t;
        const int g = r / p.Lt, pos = m * p.Lt + (r - g * p.Lt);
        if (m >= p.nM || g >= p.G || pos >= tile_end(p, m)) return;
        constexpr int U = 4;
        for (int k = c; k <= sp.w; k += U) {
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
            for (int u = 0; u < U; ++u) st.add(v[u], x[u]);
        }
        store_row(p, (static_cast<long long>(sp.x) * p.H_q + sp.y * p.G + g) * p.L + pos, lane, st.acc, st.l, st.M);
        return;
    }
    const int bk = rest, rr = warp;
    if (rr >= p.nrem) return;
    const int b = bk / p.H_kv, kvh = bk - b * p.H_kv;
    bool bad;
    const int S = seq_len(p, b, bad);
    if (bad) return;  // (its rows are zeros already)
    const int per = p.prefix[p.B], hu = head_units(p, S), ng = seg_units(p, S, p.nPairs - 1);
    const int last = p.prefix[b] + (kvh + 1) * hu - 1, first = last - ng + 1;  // its tiles' positions
    for (int k = first / per; k <= last / per; ++k)
        for (int w = 0; w < 2; ++w) {
            const long long slot = ((static_cast<long long>(bk) + k) * 2 + w) * 8 + rr;
            st.add(p.rem_ml[slot], *reinterpret_cast<const float4*>(p.rem_o + slot * kD + 4 * lane));
        }
    const int Lrem = p.L - p.rem_l0, g = rr / Lrem;
    store_row(p, (static_cast<long long>(b) * p.H_q + kvh * p.G + g) * p.L + p.rem_l0 + rr - g * Lrem, lane, st.acc, st.l,
              st.M);
}

constexpr int kMinPer = 4;  // least cost of a share

struct TilePlan {
    int G, Lt, nM, nPairs, nrem, rem_l0;
    size_t prefix_off, split_off, ml_off, o_off, rem_ml_off, rem_o_off, total;
};

TilePlan plan(const pa_shape& sh, int sm_count) {
    TilePlan t;
    t.G = sh.H_q / sh.H_kv;
    t.Lt = BM / t.G;
    t.nM = (sh.L + t.Lt - 1) / t.Lt;
    t.nrem = 0;
    t.rem_l0 = sh.L;
    const int rem = t.G * (sh.L - (t.nM - 1) * t.Lt);
    if (t.nM >= 3 && t.nM % 2 == 1 && rem <= 8) {
        t.nrem = rem;
        t.nM -= 1;
        t.rem_l0 = t.nM * t.Lt;
    }
    t.nPairs = (t.nM + 1) / 2;
    const size_t slots = 2ull * sm_count * 2 * BM;
    const size_t rem_slots = t.nrem ? (static_cast<size_t>(sh.B) * sh.H_kv + sm_count) * 2 * 8 : 0;
    size_t off = kFlagBytes;
    t.prefix_off = off;
    off = align_up(off + 4 * (static_cast<size_t>(sh.B) + 1), 256);
    t.split_off = off;
    off = align_up(off + 16ull * sm_count, 256);
    t.ml_off = off;
    off = align_up(off + slots * 8, 256);
    t.o_off = off;
    off = align_up(off + slots * kD * 4, 256);
    t.rem_ml_off = off;
    off = align_up(off + rem_slots * 8, 256);
    t.rem_o_off = off;
    t.total = align_up(off + rem_slots * kD * 4, 256);
    return t;
}

template <bool Q4, bool ONE>
pa_status launch_tiles(const TileParams& p, const WalkCall& c) {
    static int attr_done[64] = {0};
    if (!attr_done[c.dev.device]) {
        if (cudaFuncSetAttribute(tile_kernel<Q4, ONE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 smem_bytes(Q4, ONE)) != cudaSuccess)
            return PA_ERR_CUDA;
        attr_done[c.dev.device] = 1;
    }
    tile_kernel<Q4, ONE><<<static_cast<unsigned>(c.dev.sm_count), kThreads, smem_bytes(Q4, ONE), c.stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

bool tiles_supported(const pa_shape& sh, int sm_count) {
    const long long G = sh.H_q / sh.H_kv;
    if (sh.dtype != PA_BF16 || G > BM || sm_count < 1) return false;
    const long long cap = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    // units are counted in an int; a merge CTA per (sequence, kv head)
    const long long pairs = (sh.L + 2 * (BM / G) - 1) / (2 * (BM / G)) + 1;
    return static_cast<long long>(sh.B) * sh.H_kv * pairs * (cap / BN + 1 + kSegCost) < INT_MAX / 2 &&
           static_cast<long long>(sh.H_q) * sh.L * sh.B < (1ll << 31);
}

size_t tiles_workspace_bytes(const pa_shape& sh, int sm_count) { return plan(sh, sm_count).total; }
size_t tiles_workspace_most(const pa_shape& sh, int sm_count) {
    const size_t slots = 4ull * sm_count * BM, rem_slots = (static_cast<size_t>(sh.B) * sh.H_kv + sm_count) * 2 * 8;
    return kFlagBytes + 4 * (static_cast<size_t>(sh.B) + 1) + 16ull * sm_count + (slots + rem_slots) * (8 + kD * 4) + 6 * 256;
}

pa_status tiles_launch(const WalkCall& c, float* lse) {
    const pa_shape& sh = c.sh;
    if (c.dev.smem_optin < smem_bytes(true, true)) return PA_ERR_UNSUPPORTED;
    const TilePlan t = plan(sh, c.dev.sm_count);
    if (c.ws_bytes < t.total) return PA_ERR_WORKSPACE;
    uint8_t* const ws = static_cast<uint8_t*>(c.ws);
    TileParams p;
    p.q = static_cast<const uint16_t*>(c.q);
    p.kc = static_cast<const uint8_t*>(c.kc);
    p.ks = static_cast<const uint8_t*>(c.ks);
    p.vc = static_cast<const uint8_t*>(c.vc);
    p.vs = static_cast<const uint8_t*>(c.vs);
    p.bt = c.bt;
    p.ctx = c.ctx;
    p.out = static_cast<uint16_t*>(c.out);
    p.lse = lse;
    p.flag = reinterpret_cast<uint32_t*>(ws);
    p.part_ml = reinterpret_cast<float2*>(ws + t.ml_off);
    p.part_o = reinterpret_cast<float*>(ws + t.o_off);
    p.split = reinterpret_cast<int4*>(ws + t.split_off);
    p.rem_ml = reinterpret_cast<float2*>(ws + t.rem_ml_off);
    p.rem_o = reinterpret_cast<float*>(ws + t.rem_o_off);
    p.prefix = reinterpret_cast<int*>(ws + t.prefix_off);
    p.B = sh.B;
    p.H_q = sh.H_q;
    p.H_kv = sh.H_kv;
    p.L = sh.L;
    p.G = t.G;
    p.Lt = t.Lt;
    p.nM = t.nM;
    p.nPairs = t.nPairs;
    p.num_pages = sh.num_pages;
    p.ps = sh.page_size;
    p.max_npg = sh.max_pages_per_seq;
    p.causal = c.causal;
    p.nrem = t.nrem;
    p.rem_l0 = t.rem_l0;
    p.max_S = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    p.scale_log2 = c.scale * 1.4426950408889634f;
    p.min_per = kMinPer;
    p.out32 = reinterpret_cast<uintptr_t>(c.out) % 32 == 0;
    const pa_status st = t.nM > 1 ? (c.ks ? launch_tiles<true, false>(p, c) : launch_tiles<false, false>(p, c))
                                  : (c.ks ? launch_tiles<true, true>(p, c) : launch_tiles<false, true>(p, c));
    if (st != PA_OK) return st;
    const int shares = c.dev.sm_count;
    const int ny = (t.nM > 1 ? 2 : 1) * BM / kMergeRows;
    const dim3 grid(static_cast<unsigned>(shares * ny + (t.nrem ? sh.B * sh.H_kv : 0)));
    return launch_dependent(tile_merge_kernel, grid, 256, 0, c.stream, p, shares, ny) ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
