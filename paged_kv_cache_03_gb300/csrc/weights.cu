// weights.cu -- what every key received: the key weights of walk.cu's formulas, summed
// in a fixed order (no atomics).
#include "walk.cuh"

namespace pa {
namespace walk {
namespace {

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

// The packed query: the rows of every (sequence, kv head) as B fragments, [part]
// [(b, kvh)][n-tile of 8 rows][k-step pair][lane], and per row what its scores need.
struct PackedRow {
    float qs, nl;  // a product times qs is a score in log2 units; minus the log-sum-exp
};
struct Packed {
    uint4* frags;
    PackedRow* rows;  // [(b, kvh)][n-tile][8]; a row past the last one weighs 2^-inf = 0
    int* last;        // the last key a row sees
    float* part;      // [split][(b, kvh)][w_S] sums over a split of the rows
    int nt, nsplit;
};

template <class Keys, bool F32>
__global__ void __launch_bounds__(kWarps * 32) pack_query_kernel(const WalkParams p, const Packed k) {
    const long long tile = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const long long tiles = static_cast<long long>(p.B) * p.H_kv * k.nt;
    if (tile >= tiles) return;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const long long bk = tile / k.nt;
    const int r = 8 * static_cast<int>(tile - bk * k.nt) + g;
    const int S = seq_len(p, static_cast<int>(bk / p.H_kv), false);
    QueryFrags<Keys, F32> q;
    const float down = q.load(p.q, bk * p.R + r, r < p.R, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        k.frags[(tile * 4 + i) * 32 + lane] =
            make_uint4(q.hi[2 * i][0], q.hi[2 * i][1], q.hi[2 * i + 1][0], q.hi[2 * i + 1][1]);
        if constexpr (F32)
            k.frags[((tiles + tile) * 4 + i) * 32 + lane] =
                make_uint4(q.lo[2 * i][0], q.lo[2 * i][1], q.lo[2 * i + 1][0], q.lo[2 * i + 1][1]);
    }
    if (t == 0) {
        k.rows[tile * 8 + g] = {fmaxf(down * p.scale_log2, FLT_MIN), r < p.R ? -p.lse[bk * p.R + r] : neg_inf()};
        k.last[tile * 8 + g] = p.causal ? r % p.L + S - p.L : S - 1;
    }
}

// The same from the query and the keys, for many rows: a CTA takes 128 keys of
// one (sequence, kv head), each warp 32 of them as A fragments in registers, and
// runs over the packed query rows (16 bytes a lane and k-step pair, shared by its
// warps through L1), the next 8 rows requested before these are multiplied.  Bound
// by the warp-level MMA rate (8 cycles per m16n8k16 and SM sub-partition).  Few keys
// and many rows: the rows are cut into nsplit runs, whose sums add_splits_kernel adds.
template <class Keys, bool F32>
__global__ void __launch_bounds__(kWarps * 32) weights_kernel(const WalkParams p, int ntile, const Packed pk) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int tile = static_cast<int>(blockIdx.x) % ntile, bk = static_cast<int>(blockIdx.x) / ntile;
    const int b = bk / p.H_kv, kvh = bk - b * p.H_kv;
    const long long first = (static_cast<long long>(tile) * kWarps + warp) * 32;
    pdl_launch_dependents();
    pdl_wait_primary();
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
                Keys kk;
                kk.load(p, rows, u, g, t);
                const typename Keys::Scales ksc = kk.scales();
#pragma unroll
                for (int i = 0; i < 4; ++i) kk.frags(ksc, i, *reinterpret_cast<uint32_t(*)[2][4]>(a[u][2 * i]));
            }
        }
        const long long tiles = static_cast<long long>(p.B) * p.H_kv * pk.nt, mine = static_cast<long long>(bk) * pk.nt;
        const int n0 = static_cast<int>(static_cast<long long>(pk.nt) * blockIdx.y / pk.nsplit);
        const int n1 = static_cast<int>(static_cast<long long>(pk.nt) * (blockIdx.y + 1) / pk.nsplit);
        const uint4* const q0 = pk.frags + mine * 128 + lane;
        const float4* const rows = reinterpret_cast<const float4*>(pk.rows + mine * 8 + 2 * t);
        const int2* const last = reinterpret_cast<const int2*>(pk.last + mine * 8 + 2 * t);
        uint4 next[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) next[i] = __ldg(q0 + n0 * 128 + 32 * i);
        float4 row_next = __ldg(rows + n0 * 4);
        int2 lim_next = __ldg(last + n0 * 4);
        for (int n = n0; n < n1; ++n) {
            uint4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = next[i];
            const float4 row = row_next;
            const int2 lim = lim_next;
            if (n + 1 < n1) {
#pragma unroll
                for (int i = 0; i < 4; ++i) next[i] = __ldg(q0 + (n + 1) * 128 + 32 * i);
                row_next = __ldg(rows + (n + 1) * 4);
                lim_next = __ldg(last + (n + 1) * 4);
            }
            if (!__any_sync(0xffffffffu, max(lim.x, lim.y) >= k0)) continue;
            float s[2][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (i == 0)
                        mma_first<Keys::kF16>(s[u], a[u][0], x[0].x, x[0].y);
                    else
                        mma<Keys::kF16>(s[u], a[u][2 * i], x[i].x, x[i].y);
                    mma<Keys::kF16>(s[u], a[u][2 * i + 1], x[i].z, x[i].w);
                }
            if constexpr (F32) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 y = __ldg(q0 + (tiles + n) * 128 + 32 * i);
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
                    acc[u][h] += fast_exp2(fmaf(s[u][2 * h], row.x, row.y)) + fast_exp2(fmaf(s[u][2 * h + 1], row.z, row.w));
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
    if (pk.nsplit > 1) {
        pk.part[static_cast<long long>(blockIdx.y) * p.B * p.H_kv * p.w_S + at] = sum;
    } else {
        const float old = p.w_in && key < S ? p.w_in[at] : 0.f;
        p.w_out[at] = key < S ? old + sum : 0.f;
    }
}

__global__ void __launch_bounds__(256) add_splits_kernel(const WalkParams p, const float* part, int nsplit) {
    pdl_launch_dependents();
    pdl_wait_primary();
    const long long n = static_cast<long long>(p.B) * p.H_kv * p.w_S;
    for (long long at = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; at < n;
         at += static_cast<long long>(gridDim.x) * 256) {
        const long long bk = at / p.w_S;
        const bool in = at - bk * p.w_S < seq_len(p, static_cast<int>(bk / p.H_kv), false);
        float sum = 0.f;
        for (int k = 0; k < nsplit; ++k) sum += part[k * n + at];
        p.w_out[at] = in ? (p.w_in ? p.w_in[at] : 0.f) + sum : 0.f;
    }
}

// Splits of the rows: about two CTAs per SM, of at least 64 rows.
int row_splits(long long ctas, int nt, int sm_count) {
    const long long want = (2ll * sm_count + ctas - 1) / (ctas > 0 ? ctas : 1), most = (nt + 7) / 8;
    return static_cast<int>(want < most ? want : most);
}

// Bytes of the packed query but for the partial sums.
size_t packed_bytes(long long bk, int nt, bool f32) {
    return static_cast<size_t>(bk) * nt * (128 * 16 * (f32 ? 2 : 1) + 8 * (sizeof(PackedRow) + 4));
}

template <class Keys, bool F32>
pa_status launch_weights(const WalkParams& p, void* scratch, int sm_count, cudaStream_t stream) {
    const long long bk = static_cast<long long>(p.B) * p.H_kv, ntile = (p.w_S + 32 * kWarps - 1) / (32 * kWarps);
    Packed k;
    k.nt = (p.R + 7) / 8;
    if (ntile * bk > INT_MAX || bk * k.nt > INT_MAX) return PA_ERR_UNSUPPORTED;
    // counted in the table's own keys, so that the workspace does not depend on w_S
    const long long own = (p.max_S + 32 * kWarps - 1) / (32 * kWarps);
    k.nsplit = p.w_S <= own * 32 * kWarps ? row_splits(own * bk, k.nt, sm_count) : 1;
    k.frags = static_cast<uint4*>(scratch);
    k.rows = reinterpret_cast<PackedRow*>(k.frags + bk * k.nt * 128 * (F32 ? 2 : 1));
    k.last = reinterpret_cast<int*>(k.rows + bk * k.nt * 8);
    k.part = reinterpret_cast<float*>(k.last + bk * k.nt * 8);
    pack_query_kernel<Keys, F32><<<static_cast<unsigned>((bk * k.nt + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(p, k);
    if (cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
    if (!launch_dependent(weights_kernel<Keys, F32>, dim3(static_cast<unsigned>(ntile * bk), static_cast<unsigned>(k.nsplit)),
                          kWarps * 32, stream, p, static_cast<int>(ntile), k))
        return PA_ERR_CUDA;
    if (k.nsplit == 1) return PA_OK;
    const long long blocks = (bk * p.w_S + 255) / 256, most = 8ll * sm_count;
    return launch_dependent(add_splits_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), 256, stream, p,
                            static_cast<const float*>(k.part), k.nsplit)
               ? PA_OK
               : PA_ERR_CUDA;
}

}  // namespace

pa_status weights_from_scores(const WalkParams& p, cudaStream_t stream) {
    const long long bk = static_cast<long long>(p.B) * p.H_kv, ntile = (p.w_S + 255) / 256;
    if (ntile * bk > INT_MAX) return PA_ERR_UNSUPPORTED;
    return launch_dependent(walk_sum_kernel, dim3(static_cast<unsigned>(ntile * bk)), 256, stream, p,
                            static_cast<int>(ntile))
               ? PA_OK
               : PA_ERR_CUDA;
}

size_t weights_scratch_bytes(const pa_shape& sh, int sm_count) {
    const long long bk = static_cast<long long>(sh.B) * sh.H_kv;
    const int nt = static_cast<int>((static_cast<long long>(sh.H_q / sh.H_kv) * sh.L + 7) / 8);
    const long long cap = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    const long long own = (cap + 32 * kWarps - 1) / (32 * kWarps);
    const int nsplit = row_splits(own * bk, nt, sm_count);
    return packed_bytes(bk, nt, sh.dtype == PA_F32) +
           (nsplit > 1 ? static_cast<size_t>(nsplit) * bk * own * 32 * kWarps * 4 : 0);
}

pa_status weights_from_keys(const WalkParams& p, bool q4, bool f32, void* scratch, int sm_count, cudaStream_t stream) {
    if (!q4) return launch_weights<BfKeys, false>(p, scratch, sm_count, stream);
    return f32 ? launch_weights<Q4Keys, true>(p, scratch, sm_count, stream)
               : launch_weights<Q4Keys, false>(p, scratch, sm_count, stream);
}

}  // namespace walk
}  // namespace pa
