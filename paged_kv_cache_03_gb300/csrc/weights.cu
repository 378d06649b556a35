// weights.cu -- what every key received: the key weights of walk.cu's formulas, summed
// in a fixed order (no atomics).
#include "walk.cuh"

namespace pa {
namespace walk {
namespace {

constexpr int kSumKeys = 4;  // keys of a thread of walk_sum_kernel

// A row's weight of a key from the score in log2 units, 0 for one it does not see (-inf; the
// row's log-sum-exp may be NaN).
__device__ __forceinline__ float weight_of(float score, float lse) {
    return score == neg_inf() ? 0.f : fast_exp2(score - lse);
}
__device__ __forceinline__ float weight_of(float product, float scale, float minus_lse) {
    return product == neg_inf() ? 0.f : fast_exp2(fmaf(product, scale, minus_lse));
}

// w_out[b, kvh, k] = w_in[b, kvh, k] + the rows' probabilities of key k, 0 past
// the context, from the scores that walk_kernel left.  Four keys per thread, 256
// apart, their loads together (64 sequences of 128 .. 4096 4-bit keys, 4 rows, the call:
// 65 us with one key a thread, 60 with four); the R scores of a key lie together, so a
// warp reads them as whole lines.  Bound by the scores read and the weights' lines.
__global__ void __launch_bounds__(256) walk_sum_kernel(const WalkParams p, int ntile) {
    const int tile = static_cast<int>(blockIdx.x) % ntile;
    const long long bk = static_cast<int>(blockIdx.x) / ntile;
    const long long k0 = static_cast<long long>(tile) * (256 * kSumKeys) + threadIdx.x;
    pdl_wait_primary();
    const int S = seq_len(p, static_cast<int>(bk / p.H_kv), false);
    const float* const x = p.score + bk * p.cap * p.R;
    const float* const lse = p.lse + bk * p.R;
    float acc[kSumKeys] = {}, old[kSumKeys] = {};
#pragma unroll
    for (int j = 0; j < kSumKeys; ++j)
        if (p.w_in && k0 + 256 * j < S) old[j] = p.w_in[bk * p.w_S + k0 + 256 * j];
    if (p.R % 4 == 0) {
        for (int r = 0; r < p.R; r += 4) {
            float4 v[kSumKeys];
#pragma unroll
            for (int j = 0; j < kSumKeys; ++j)
                if (k0 + 256 * j < S) v[j] = *reinterpret_cast<const float4*>(x + (k0 + 256 * j) * p.R + r);
            const float l[4] = {lse[r], lse[r + 1], lse[r + 2], lse[r + 3]};
#pragma unroll
            for (int j = 0; j < kSumKeys; ++j) {
                if (k0 + 256 * j >= S) continue;
                acc[j] += weight_of(v[j].x, l[0]);
                acc[j] += weight_of(v[j].y, l[1]);
                acc[j] += weight_of(v[j].z, l[2]);
                acc[j] += weight_of(v[j].w, l[3]);
            }
        }
    } else {
        for (int r = 0; r < p.R; ++r) {
            const float l = lse[r];
#pragma unroll
            for (int j = 0; j < kSumKeys; ++j)
                if (k0 + 256 * j < S) acc[j] += weight_of(x[(k0 + 256 * j) * p.R + r], l);
        }
    }
#pragma unroll
    for (int j = 0; j < kSumKeys; ++j) {
        const long long k = k0 + 256 * j;
        if (k < p.w_S) p.w_out[bk * p.w_S + k] = k < S ? acc[j] + old[j] : 0.f;
    }
}

// The packed query: the rows of every (sequence, kv head) as B fragments, [part]
// [(b, kvh)][n-tile of 8 rows][k-step pair][lane], and per row what its scores need.
struct PackedRow {
    float qs, nl;  // a product times qs is a score in log2 units; minus the log-sum-exp
};
struct Packed {
    uint4* frags;
    PackedRow* rows;  // [(b, kvh)][n-tile][8]; a row past the last one weighs 2^-inf = 0
    int* last;        // the last key a row sees
    int nt;
};

__global__ void __launch_bounds__(kWarps * 32) pack_query_kernel(const WalkParams p, const Packed k) {
    const long long tile = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const long long tiles = static_cast<long long>(p.B) * p.H_kv * k.nt;
    if (tile >= tiles) return;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const long long bk = tile / k.nt;
    const int r = 8 * static_cast<int>(tile - bk * k.nt) + g;
    const int S = seq_len(p, static_cast<int>(bk / p.H_kv), false);
    QueryFrags<Q4Keys, true> q;
    const float down = q.load(p.q, bk * p.R + r, r < p.R, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        k.frags[(tile * 4 + i) * 32 + lane] =
            make_uint4(q.hi[2 * i][0], q.hi[2 * i][1], q.hi[2 * i + 1][0], q.hi[2 * i + 1][1]);
        k.frags[((tiles + tile) * 4 + i) * 32 + lane] =
            make_uint4(q.lo[2 * i][0], q.lo[2 * i][1], q.lo[2 * i + 1][0], q.lo[2 * i + 1][1]);
    }
    if (t == 0) {
        k.rows[tile * 8 + g] = {fmaxf(down * p.scale_log2, FLT_MIN), r < p.R ? -p.lse[bk * p.R + r] : neg_inf()};
        k.last[tile * 8 + g] = p.causal ? r % p.L + S - p.L : S - 1;
    }
}

// The same from an fp32 query and 4-bit keys, for many rows: a CTA takes 128 keys of
// one (sequence, kv head), each warp 32 of them as A fragments in registers, and
// runs over the packed query rows (16 bytes a lane and k-step pair, shared by its
// warps through L1), the next 8 rows requested before these are multiplied.  Bound
// by the warp-level MMA rate (8 cycles per m16n8k16 and SM sub-partition).  Few keys
// and many rows: the rows are cut into runs, whose sums add_splits_kernel adds (with bf16
// rows then: 7 heads x 196 rows over 196 keys 90 us without runs, 39 with).
__global__ void __launch_bounds__(kWarps * 32) weights_kernel(const WalkParams p, int ntile, const Packed pk,
                                                              const RowSplits sp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int tile = static_cast<int>(blockIdx.x) % ntile, bk = static_cast<int>(blockIdx.x) / ntile;
    const int b = bk / p.H_kv, kvh = bk - b * p.H_kv;
    const long long first = (static_cast<long long>(tile) * kWarps + warp) * 32;
    pdl_launch_dependents();
    pdl_wait_primary();
    // (the packed query is the kernel before's: plain loads, which stay behind the wait)
    const int S = seq_len(p, b, false);
    float acc[2][2] = {};  // keys g and g + 8 of both halves, this lane's rows
    if (first < S) {       // (uniform over the warp)
        const int k0 = static_cast<int>(first);
        uint32_t a[2][8][4];
        {
            StepWalker<false, 2> wk;
            wk.start(p, k0 + lane, 0);
            int pg[2];
            wk.pages(p.bt + static_cast<long long>(b) * p.max_npg, p, k0 + lane < S ? INT_MAX : 0, pg);
            const StepRows<false, 2> rows = wk.rows(p, kvh, pg);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                Q4Keys kk;
                kk.load(p, rows, u, g, t);
                const Q4Keys::Scales ksc = kk.scales();
#pragma unroll
                for (int i = 0; i < 4; ++i) kk.frags(ksc, i, *reinterpret_cast<uint32_t(*)[2][4]>(a[u][2 * i]));
            }
        }
        const long long tiles = static_cast<long long>(p.B) * p.H_kv * pk.nt, mine = static_cast<long long>(bk) * pk.nt;
        const int n0 = static_cast<int>(static_cast<long long>(pk.nt) * blockIdx.y / sp.n);
        const int n1 = static_cast<int>(static_cast<long long>(pk.nt) * (blockIdx.y + 1) / sp.n);
        const uint4* const q0 = pk.frags + mine * 128 + lane;
        const float4* const rows = reinterpret_cast<const float4*>(pk.rows + mine * 8 + 2 * t);
        const int2* const last = reinterpret_cast<const int2*>(pk.last + mine * 8 + 2 * t);
        uint4 next[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) next[i] = q0[n0 * 128 + 32 * i];
        float4 row_next = rows[n0 * 4];
        int2 lim_next = last[n0 * 4];
        for (int n = n0; n < n1; ++n) {
            uint4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = next[i];
            const float4 row = row_next;
            const int2 lim = lim_next;
            if (n + 1 < n1) {
#pragma unroll
                for (int i = 0; i < 4; ++i) next[i] = q0[(n + 1) * 128 + 32 * i];
                row_next = rows[(n + 1) * 4];
                lim_next = last[(n + 1) * 4];
            }
            if (!__any_sync(0xffffffffu, max(lim.x, lim.y) >= k0)) continue;
            float s[2][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (i == 0)
                        mma_first<true>(s[u], a[u][0], x[0].x, x[0].y);
                    else
                        mma<true>(s[u], a[u][2 * i], x[i].x, x[i].y);
                    mma<true>(s[u], a[u][2 * i + 1], x[i].z, x[i].w);
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 y = q0[(tiles + n) * 128 + 32 * i];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    mma<true>(s[u], a[u][2 * i], y.x, y.y);
                    mma<true>(s[u], a[u][2 * i + 1], y.z, y.w);
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
                    acc[u][h] += weight_of(s[u][2 * h], row.x, row.y) + weight_of(s[u][2 * h + 1], row.z, row.w);
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
    const float sum = t & 2 ? (t & 1 ? acc[1][1] : acc[1][0]) : (t & 1 ? acc[0][1] : acc[0][0]);
    const long long key = first + 16 * (t >> 1) + g + 8 * (t & 1);
    if (key >= p.w_S) return;
    const long long at = static_cast<long long>(bk) * p.w_S + key;
    if (sp.n > 1) {
        if (key < S) sp.at(p, blockIdx.y, bk)[key] = sum;
    } else {
        const float old = p.w_in && key < S ? p.w_in[at] : 0.f;
        p.w_out[at] = key < S ? old + sum : 0.f;
    }
}

__global__ void __launch_bounds__(256) add_splits_kernel(const WalkParams p, const RowSplits sp) {
    pdl_launch_dependents();
    pdl_wait_primary();
    const long long n = static_cast<long long>(p.B) * p.H_kv * p.w_S;
    for (long long at = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; at < n;
         at += static_cast<long long>(gridDim.x) * 256) {
        const int bk = static_cast<int>(at / p.w_S);
        const long long key = at - bk * p.w_S;
        float sum = 0.f;
        if (key < seq_len(p, bk / p.H_kv, false)) {
            for (int k = 0; k < sp.n; ++k) sum += sp.at(p, k, bk)[key];
            if (p.w_in) sum += p.w_in[at];
        }
        p.w_out[at] = sum;
    }
}

constexpr int kKeysCta = 32 * kWarps;  // keys of a CTA that recomputes

// How the rows are cut: about two CTAs per SM, of at least 64 rows.  (Counted in the
// table's keys, so that neither the workspace nor the sums depend on w_S.)
int row_runs(long long bk, long long cap, int R, int sm_count) {
    const long long ctas = bk * ((cap + kKeysCta - 1) / kKeysCta), most = (R + 63) / 64;
    const long long want = (2ll * sm_count + ctas - 1) / (ctas > 0 ? ctas : 1);
    return static_cast<int>(want < most ? want : most);
}
size_t runs_bytes(long long bk, long long cap, int R, int sm_count) {
    const int n = row_runs(bk, cap, R, sm_count);
    return n > 1 ? align_up(static_cast<size_t>(n) * bk * cap * 4, 16) : 0;
}
// fp32 queries (over 4-bit pages).
pa_status weights_of_f32(const WalkParams& p, const RowSplits& sp, void* scratch, cudaStream_t stream) {
    const long long bk = static_cast<long long>(p.B) * p.H_kv, ntile = (p.w_S + kKeysCta - 1) / kKeysCta;
    Packed k;
    k.nt = (p.R + 7) / 8;
    k.frags = static_cast<uint4*>(scratch);
    k.rows = reinterpret_cast<PackedRow*>(k.frags + bk * k.nt * 256);
    k.last = reinterpret_cast<int*>(k.rows + bk * k.nt * 8);
    pack_query_kernel<<<static_cast<unsigned>((bk * k.nt + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(p, k);
    if (cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
    const dim3 grid(static_cast<unsigned>(ntile * bk), static_cast<unsigned>(sp.n));
    return launch_dependent(weights_kernel, grid, kWarps * 32, 0, stream, p, static_cast<int>(ntile), k, sp) ? PA_OK
                                                                                                            : PA_ERR_CUDA;
}

}  // namespace

pa_status weights_from_scores(const WalkParams& p, cudaStream_t stream) {
    const long long bk = static_cast<long long>(p.B) * p.H_kv, ntile = (p.w_S + 256 * kSumKeys - 1) / (256 * kSumKeys);
    return launch_dependent(walk_sum_kernel, dim3(static_cast<unsigned>(ntile * bk)), 256, 0, stream, p,
                            static_cast<int>(ntile))
               ? PA_OK
               : PA_ERR_CUDA;
}

bool weights_supported(const pa_shape& sh, long long w_S, int sm_count) {
    const long long bk = static_cast<long long>(sh.B) * sh.H_kv, cap = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    const long long R = static_cast<long long>(sh.H_q / sh.H_kv) * sh.L;
    // items and blocks are counted in ints, and so are a kv head's query tiles times 128
    if (R >= (1ll << 27)) return false;
    const long long most = INT_MAX / 2 / bk / row_runs(bk, cap, static_cast<int>(R), sm_count);
    return w_S <= INT_MAX / 2 && w_S / kKeysCta < most && bk * ((R + 7) / 8) <= INT_MAX;
}

// The packed query of fp32 calls.
static size_t packed_bytes(const pa_shape& sh) {
    const size_t tile = 2 * 128 * 16 + 8 * (sizeof(PackedRow) + sizeof(int));
    const long long R = static_cast<long long>(sh.H_q / sh.H_kv) * sh.L;
    return sh.dtype == PA_F32 ? static_cast<size_t>(sh.B) * sh.H_kv * ((R + 7) / 8) * tile : 0;
}

size_t weights_scratch_bytes(const pa_shape& sh, int sm_count) {
    const long long bk = static_cast<long long>(sh.B) * sh.H_kv;
    const long long R = static_cast<long long>(sh.H_q / sh.H_kv) * sh.L;
    const long long cap = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    return runs_bytes(bk, cap, static_cast<int>(R), sm_count) + packed_bytes(sh);
}

size_t weights_scratch_most(const pa_shape& sh, int sm_count) {
    // runs: two CTAs an SM and the CTAs of one run, themselves less than that, 128 keys each
    return 4ull * sm_count * kKeysCta * 4 + 16 + packed_bytes(sh);
}

pa_status weights_from_keys(const WalkParams& p, bool q4, bool f32, void* scratch, const DeviceInfo& dev,
                            cudaStream_t stream) {
    const long long bk = static_cast<long long>(p.B) * p.H_kv;
    const RowSplits sp = {static_cast<float*>(scratch), row_runs(bk, p.max_S, p.R, dev.sm_count)};
    void* const packed = static_cast<uint8_t*>(scratch) + runs_bytes(bk, p.max_S, p.R, dev.sm_count);
    const pa_status st = f32 ? weights_of_f32(p, sp, packed, stream) : weights_on_tiles(p, q4, sp, dev, stream);
    if (st != PA_OK || sp.n == 1) return st;
    const long long blocks = (bk * p.w_S + 255) / 256, most = 8ll * dev.sm_count;
    return launch_dependent(add_splits_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), 256, 0, stream, p, sp)
               ? PA_OK
               : PA_ERR_CUDA;
}

}  // namespace walk
}  // namespace pa
