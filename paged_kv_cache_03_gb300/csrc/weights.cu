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

// The query rows of every (sequence, kv head) as B fragments, 8 rows a warp: [part]
// [(b, kvh)][n-tile][k-step pair][lane], and what takes a product with them to a
// score in log2 units.
template <class Keys, bool F32>
__global__ void __launch_bounds__(kWarps * 32) pack_query_kernel(const WalkParams p, int nt, uint4* frags, float* scale) {
    const long long tile = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const long long tiles = static_cast<long long>(p.B) * p.H_kv * nt;
    if (tile >= tiles) return;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const long long bk = tile / nt;
    const int r = 8 * static_cast<int>(tile - bk * nt) + g;
    QueryFrags<Keys, F32> q;
    const float down = q.load(p.q, bk * p.R + r, r < p.R, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        frags[(tile * 4 + i) * 32 + lane] = make_uint4(q.hi[2 * i][0], q.hi[2 * i][1], q.hi[2 * i + 1][0], q.hi[2 * i + 1][1]);
        if constexpr (F32)
            frags[((tiles + tile) * 4 + i) * 32 + lane] =
                make_uint4(q.lo[2 * i][0], q.lo[2 * i][1], q.lo[2 * i + 1][0], q.lo[2 * i + 1][1]);
    }
    if (t == 0) scale[tile * 8 + g] = fmaxf(down * p.scale_log2, FLT_MIN);
}

// The same from the query and the keys, for many rows: a CTA takes 128 keys of
// one (sequence, kv head), each warp 32 of them as A fragments in registers, and
// runs over the packed query rows (16 bytes a lane and k-step pair, shared by its
// warps through L1), the next 8 rows requested before these are multiplied.  Bound
// by the warp-level MMA rate (8 cycles per m16n8k16 and SM sub-partition).
template <class Keys, bool F32>
__global__ void __launch_bounds__(kWarps * 32) weights_kernel(const WalkParams p, int ntile, int nt, const uint4* frags,
                                                             const float* scale) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int tile = static_cast<int>(blockIdx.x) % ntile, bk = static_cast<int>(blockIdx.x) / ntile;
    const int b = bk / p.H_kv, kvh = bk - b * p.H_kv;
    const long long first = (static_cast<long long>(tile) * kWarps + warp) * 32;
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
        const long long tiles = static_cast<long long>(p.B) * p.H_kv * nt, mine = static_cast<long long>(bk) * nt;
        const uint4* const q0 = frags + mine * 128 + lane;
        const float* const sc = scale + mine * 8 + 2 * t;
        const float* const lse = p.lse + static_cast<long long>(bk) * p.R;
        uint4 next[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) next[i] = __ldg(q0 + 32 * i);
        for (int n = 0; n < nt; ++n) {
            uint4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = next[i];
            if (n + 1 < nt) {
#pragma unroll
                for (int i = 0; i < 4; ++i) next[i] = __ldg(q0 + (n + 1) * 128 + 32 * i);
            }
            const int r = 8 * n + 2 * t;
            int lim[2] = {S - 1, S - 1};
            if (p.causal) {
                lim[0] = r % p.L + S - p.L;
                lim[1] = (r + 1) % p.L + S - p.L;
            }
            if (!__any_sync(0xffffffffu, max(lim[0], lim[1]) >= k0)) continue;
            const float2 qs = __ldg(reinterpret_cast<const float2*>(sc + 8 * n));
            // (a row past the last one weighs 2^-inf = 0)
            const float l0 = r < p.R ? lse[r] : __int_as_float(0x7f800000);
            const float l1 = r + 1 < p.R ? lse[r + 1] : __int_as_float(0x7f800000);
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
                    const uint4 y = __ldg(q0 + tiles * 128 + n * 128 + 32 * i);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        mma<Keys::kF16>(s[u], a[u][2 * i], y.x, y.y);
                        mma<Keys::kF16>(s[u], a[u][2 * i + 1], y.z, y.w);
                    }
                }
            }
            if (__any_sync(0xffffffffu, k0 + 31 > min(lim[0], lim[1]))) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (k0 + 16 * u + g + 8 * (e >> 1) > lim[e & 1]) s[u][e] = neg_inf();
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    acc[u][h] += fast_exp2(fmaf(s[u][2 * h], qs.x, -l0)) + fast_exp2(fmaf(s[u][2 * h + 1], qs.y, -l1));
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
    const long long k = first + 16 * (t >> 1) + g + 8 * (t & 1);
    if (k < p.w_S) {
        const long long at = static_cast<long long>(bk) * p.w_S + k;
        const float old = p.w_in && k < S ? p.w_in[at] : 0.f;
        p.w_out[at] = k < S ? old + sum : 0.f;
    }
}

template <class Keys, bool F32>
pa_status launch_weights(const WalkParams& p, void* scratch, cudaStream_t stream) {
    const long long bk = static_cast<long long>(p.B) * p.H_kv, ntile = (p.w_S + 32 * kWarps - 1) / (32 * kWarps);
    const int nt = (p.R + 7) / 8;
    if (ntile * bk > INT_MAX || bk * nt > INT_MAX) return PA_ERR_UNSUPPORTED;
    uint4* const frags = static_cast<uint4*>(scratch);
    float* const scale = reinterpret_cast<float*>(frags + bk * nt * 128 * (F32 ? 2 : 1));
    pack_query_kernel<Keys, F32><<<static_cast<unsigned>((bk * nt + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(
        p, nt, frags, scale);
    if (cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
    return launch_dependent(weights_kernel<Keys, F32>, dim3(static_cast<unsigned>(ntile * bk)), kWarps * 32, stream, p,
                            static_cast<int>(ntile), nt, static_cast<const uint4*>(frags),
                            static_cast<const float*>(scale))
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

size_t weights_scratch_bytes(const pa_shape& sh) {
    const size_t nt = (static_cast<size_t>(sh.H_q / sh.H_kv) * sh.L + 7) / 8, parts = sh.dtype == PA_F32 ? 2 : 1;
    return static_cast<size_t>(sh.B) * sh.H_kv * nt * (128 * 16 * parts + 8 * 4);
}

pa_status weights_from_keys(const WalkParams& p, bool q4, bool f32, void* scratch, cudaStream_t stream) {
    if (!q4) return launch_weights<BfKeys, false>(p, scratch, stream);
    return f32 ? launch_weights<Q4Keys, true>(p, scratch, stream) : launch_weights<Q4Keys, false>(p, scratch, stream);
}

}  // namespace walk
}  // namespace pa
