// weights_tiles.cu -- key weights of more than kScoreRows bf16 query rows on tcgen05
// tensor cores: the weights of walk.cu's formulas, recomputed from the query, the keys
// and the rows' log-sum-exp.
//
// An item is 128 keys of one (sequence, kv head) and a run of its query rows, 64 at a
// time: S^T = K Q^T with the keys on the MMA's M side, so that a thread reads one key's
// scores from TMEM and sums 2^(score - lse) over the rows in a register, with no shuffle
// and no atomic.  The keys stay in shared memory (4-bit rows dequantised to bf16, exact);
// query tiles come by 16-byte asynchronous copies into two buffers, and the products of
// a tile run while the tile before it is summed.  Three CTAs on an SM take the items in
// turn, the next item's 4-bit rows in registers before this one's sums: a CTA per item
// spent most of its time on its start (8 x 4 heads x 32 rows over 1000 .. 8000 keys, 8 kv
// heads: 59 us with a CTA per item, 36 so).  Items cycle over the heads first: over the
// tiles first, a CTA met the same part of every sequence (50 us).  Bound by instruction
// latency: 12 warps an SM, a key and row costing a multiply-add, an exponential and an add.
#include "stage.cuh"
#include "tc.cuh"
#include "walk.cuh"

namespace pa {
namespace walk {
namespace {

constexpr int kKeys = 128, kRows = 64, kThreads = 128;
constexpr int kQHalf = kRows * 128;  // 64 rows x 64 dims, one swizzled column block
constexpr int kOffQ = 2 * kStageHalf, kSmem = kOffQ + 2 * 2 * kQHalf + 1024;  // slack to align the base
constexpr uint32_t kCols = 2 * kRows;


// 128 keys of a (sequence, kv head) and a run of its rows.
struct Item {
    int id;  // (run * ntile + tile) * B * H_kv + bk: a CTA meets short and long sequences in turn
    int S, b, bk, run, k0;
};
// Query rows 64 n .. of a (sequence, kv head), the first at position l of its head.
struct RowTile {
    int n, l;
};

template <bool Q4>
__global__ void __launch_bounds__(kThreads, 3) weights_tile_kernel(const WalkParams p, int ntile, const RowSplits sp) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(16) float lse_s[3][kRows];
    __shared__ __align__(16) int last_s[3][kRows];  // the last key a row sees
    __shared__ __align__(8) uint64_t done_s[3];  // the products of even and odd tiles, of all at a time-out
    __shared__ uint32_t tmem_s;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int heads = p.B * p.H_kv, items = ntile * heads * sp.n;
    pdl_launch_dependents();

    // The first item at or after `id` of this CTA that has keys; the others' weights are 0.
    auto find = [&](int id) {
        Item it = {};
        for (; id < items; id += static_cast<int>(gridDim.x)) {
            const int u = id / heads;
            it.bk = id - u * heads;
            it.run = u / ntile;
            it.k0 = (u - it.run * ntile) * kKeys;
            it.b = it.bk / p.H_kv;
            it.S = seq_len(p, it.b, false);
            if (it.k0 < it.S) break;
            if (sp.n == 1 && it.k0 + tid < p.w_S) p.w_out[it.bk * p.w_S + it.k0 + tid] = 0.f;
        }
        it.id = id;
        return it;
    };
    // lane 8 i + r looks up key 32 i + 8 warp + r
    int page = kNoPage, in_page = 0;
    bool bad = false;
    auto lookup = [&](const Item& it) {
        const int k = it.k0 + 32 * (lane >> 3) + 8 * warp + (lane & 7);
        const int lp = k / p.ps;
        in_page = k - lp * p.ps;
        page = k < it.S ? __ldg(p.bt + static_cast<long long>(it.b) * p.max_npg + lp) : kNoPage;
    };
    RawTile raw;
    int rows;  // pool rows of the next item's keys
    const uint8_t* const keys = static_cast<const uint8_t*>(p.kc);
    auto request = [&](const Item& it) {
        rows = row_in(p, it.bk - it.b * p.H_kv, page, in_page, bad);
        if constexpr (Q4) raw.request(keys, static_cast<const uint8_t*>(p.ks), rows, lane);
    };

    pdl_wait_primary();  // (what follows writes the weights)
    Item it = find(static_cast<int>(blockIdx.x));
    if (it.id >= items) return;
    lookup(it);
    request(it);
    if (tid == 0) {
        mbar_init(smem_u32(&done_s[0]), 1);
        mbar_init(smem_u32(&done_s[1]), 1);
        mbar_init(smem_u32(&done_s[2]), 1);
        fence_mbar_init();
    }
    __syncwarp();
    if (warp == 0) {
        tc::tmem_alloc(smem_u32(&tmem_s), kCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_s;
    const int c = tid & 15, r0 = tid >> 4;  // this thread's 16-byte chunk, and its first row of eight
    const float scale = fmaxf(p.scale_log2, FLT_MIN);
    const int nt = (p.R + kRows - 1) / kRows, step = kRows % p.L;
    auto product = [&](int i) {
        constexpr uint32_t idesc = tc::idesc_bf16(kKeys, kRows, 0, 0);  // both K-major
        const uint64_t dk = tc::smem_desc_sw128(base, 16, 1024);
        const uint64_t dq = tc::smem_desc_sw128(base + kOffQ + (i & 1) * (2 * kQHalf), 16, 1024);
        const uint32_t d = tmem + (i & 1) * kRows;
        tc::mma_bf16_c<0>(d, dk, dq, idesc);
#pragma unroll
        for (int kk = 1; kk < kD / 16; ++kk)
            tc::mma_bf16_c<1>(d, tc::desc_advance(dk, (kk >> 2) * kStageHalf + (kk & 3) * 32),
                              tc::desc_advance(dq, (kk >> 2) * kQHalf + (kk & 3) * 32), idesc);
        tc::commit(smem_u32(&done_s[i & 1]));
    };

    bool ok = true;
    int i = 0;  // query tiles so far
    while (ok && it.id < items) {
        const long long at = static_cast<long long>(it.bk) * p.w_S + it.k0 + tid;
        const bool mine = it.k0 + tid < it.S;
        float old = 0.f;
        if (p.w_in && mine && sp.n == 1) old = p.w_in[at];
        // ---- the query tiles; one that wraps from a head to the next sees every key ------
        const int n0 = nt * it.run / sp.n;
        const int n1 = nt * (it.run + 1) / sp.n;
        auto behind = [&](RowTile x) { return RowTile{x.n + 1, x.l + step >= p.L ? x.l + step - p.L : x.l + step}; };
        auto from = [&](RowTile x) {  // the first tile at or after x that sees one of the keys
            if (p.causal)
                while (x.n < n1 && x.l + kRows <= p.L && x.l + kRows - 1 + it.S - p.L < it.k0) x = behind(x);
            return x;
        };
        auto edge = [&](RowTile x) {  // some row does not see all the keys
            return p.causal && it.k0 + kKeys - 1 > (x.l + kRows > p.L ? 0 : x.l) + it.S - p.L;
        };
        const uint16_t* const q = static_cast<const uint16_t*>(p.q) + static_cast<long long>(it.bk) * p.R * kD;
        auto fetch = [&](RowTile x, int i) {  // tile x as the i-th
            const uint32_t dst = base + kOffQ + (i & 1) * (2 * kQHalf) + (c >> 3) * kQHalf;
#pragma unroll
            for (int j = 0; j < kRows / 8; ++j) {
                const int r = x.n * kRows + r0 + 8 * j;
                cp_async16(dst + sw128(r0 + 8 * j, c & 7), q + (r < p.R ? static_cast<long long>(r) * kD : 0) + 8 * c, r < p.R);
            }
            if (tid < kRows) {
                const int r = x.n * kRows + tid;
                if (r < p.R)
                    cp_async4(smem_u32(&lse_s[i % 3][tid]), p.lse + static_cast<long long>(it.bk) * p.R + r);
                else
                    lse_s[i % 3][tid] = __int_as_float(0x7f800000);  // 2^-inf = 0
                if (edge(x)) last_s[i % 3][tid] = r % p.L + it.S - p.L;
            }
            cp_async_commit();
        };
        // ---- the keys; the next item's page ids -------------------------------------
        if constexpr (!Q4) {
            copy_tile(base, keys, rows, warp, lane);
            cp_async_commit();
        }
        RowTile now = from({n0, n0 > 0 ? n0 * kRows % p.L : 0}), next = from(behind(now));
        if (now.n < n1) fetch(now, i);
        if (next.n < n1) fetch(next, i + 1);
        const Item then = find(it.id + static_cast<int>(gridDim.x));
        if (then.id < items) lookup(then);
        if constexpr (Q4) raw.store<true>(base, warp, lane);
        if (next.n < n1)
            cp_async_wait<1>();
        else
            cp_async_wait<0>();
        fence_proxy_async_smem();
        tc::fence_before_sync();
        __syncthreads();
        tc::fence_after_sync();
        if (tid == 0 && now.n < n1) product(i);
        if (then.id < items) request(then);
        // ---- the rows ---------------------------------------------------------------
        float acc[4] = {};
        for (; now.n < n1; ++i) {
            if (next.n < n1) {
                cp_async_wait<0>();
                fence_proxy_async_smem();
            }
            tc::fence_before_sync();
            // every thread has read tile i - 1's scores, and its part of tile i + 1 is here
            if (__syncthreads_or(!ok)) {
                ok = false;
                break;
            }
            tc::fence_after_sync();
            if (tid == 0 && next.n < n1) product(i + 1);
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&done_s[i & 1]), (i >> 1) & 1));
            tc::fence_after_sync();
            const RowTile after = from(behind(next));
            if (ok && after.n < n1) fetch(after, i + 2);  // (the products have read tile i)
            const bool masked = edge(now);
            const float* const lse = lse_s[i % 3];
            const int* const last = last_s[i % 3];
#pragma unroll
            for (int h = 0; h < kRows / 32; ++h) {
                if (now.n * kRows + 32 * h >= p.R) break;  // (uniform)
                float s[32];
                tc::ld32(tmem + (static_cast<uint32_t>(32 * warp) << 16) + (i & 1) * kRows + 32 * h, s);
                tc::wait_ld();
                const int k = it.k0 + tid;
                auto add = [&](int j, float x, float m) { acc[j] += fast_exp2(fmaf(x, scale, -m)); };
                if (masked) {  // (a row that does not see the key adds nothing, whatever its sum is)
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const int4 x = *reinterpret_cast<const int4*>(last + 32 * h + e);
                        const float4 m = *reinterpret_cast<const float4*>(lse + 32 * h + e);
                        if (k <= x.x) add(0, s[e], m.x);
                        if (k <= x.y) add(1, s[e + 1], m.y);
                        if (k <= x.z) add(2, s[e + 2], m.z);
                        if (k <= x.w) add(3, s[e + 3], m.w);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 m = *reinterpret_cast<const float4*>(lse + 32 * h + e);
                        add(0, s[e], m.x);
                        add(1, s[e + 1], m.y);
                        add(2, s[e + 2], m.z);
                        add(3, s[e + 3], m.w);
                    }
                }
            }
            now = next;
            next = after;
        }
        // A wait that ran out ends the call for the whole CTA, before anything is added to the
        // weights: the warps would part at the next item's barriers otherwise.
        ok = !__syncthreads_or(!ok);
        if (!ok) break;
        const float sum = (acc[0] + acc[1]) + (acc[2] + acc[3]);
        if (sp.n > 1) {
            if (mine) sp.at(p, it.run, it.bk)[it.k0 + tid] = sum;
        } else if (it.k0 + tid < p.w_S) {
            p.w_out[at] = mine ? old + sum : 0.f;
        }
        it = then;
    }
    // (runs that are joined later: what was not summed adds nothing)
    if (!ok && sp.n > 1)
        for (it = find(it.id); it.id < items; it = find(it.id + static_cast<int>(gridDim.x)))
            if (it.k0 + tid < it.S) sp.at(p, it.run, it.bk)[it.k0 + tid] = 0.f;
    // nothing of ours may still be running when TMEM is freed
    cp_async_wait<0>();
    if (!ok && tid == 0) {
        atomicOr(p.flag, PA_FLAG_TIMEOUT);
        tc::commit(smem_u32(&done_s[2]));
        mbar_wait(smem_u32(&done_s[2]), 0);
    }
    report_pages(p, bad);
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) tc::tmem_dealloc(tmem, kCols);
}

template <bool Q4>
pa_status launch_tiles(const WalkParams& p, const RowSplits& sp, int device, int sm_count, cudaStream_t stream) {
    static int attr_done[64] = {0};
    if (!attr_done[device]) {
        if (cudaFuncSetAttribute(weights_tile_kernel<Q4>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
            return PA_ERR_CUDA;
        attr_done[device] = 1;
    }
    const long long ntile = (p.w_S + kKeys - 1) / kKeys, all = ntile * p.B * p.H_kv * sp.n, most = 3ll * sm_count;
    const dim3 grid(static_cast<unsigned>(all < most ? all : most));
    return launch_dependent(weights_tile_kernel<Q4>, grid, kThreads, kSmem, stream, p, static_cast<int>(ntile), sp)
               ? PA_OK
               : PA_ERR_CUDA;
}

}  // namespace

pa_status weights_on_tiles(const WalkParams& p, bool q4, const RowSplits& sp, const DeviceInfo& dev,
                           cudaStream_t stream) {
    return q4 ? launch_tiles<true>(p, sp, dev.device, dev.sm_count, stream)
              : launch_tiles<false>(p, sp, dev.device, dev.sm_count, stream);
}

}  // namespace walk
}  // namespace pa
