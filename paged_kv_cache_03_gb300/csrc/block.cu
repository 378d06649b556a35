// block.cu -- attention of many rows where the tensor-core tiles of tiles.cu do not
// apply: fp32 queries over 4-bit pages, bf16 pages with key weights.  The formulas and
// roundings are those of walk.cu.
//
// With more rows than a warp holds, dequantising per warp would cost more than
// the products.  Here a CTA's four warps take 16 rows each (M = rows) and the
// 64-key K and V tiles go through shared memory once, as f16 (4-bit pages) or
// as they are (bf16): S = Q K^T with K by ldmatrix, O += P V with V by
// ldmatrix.trans.  Two buffers: the next tile is requested when a tile begins
// and, 4-bit, written dequantised when it ends.  A 256-byte row holds its even
// 16-byte chunks first, then the odd ones, both permuted by the row's low bits:
// the writers (32 bytes a lane) and ldmatrix meet no bank conflict.
//
// Bound by the warp-level products, twice as many for fp32's two parts: 64 fp32 rows
// over 8 sequences of 1000 .. 8000 4-bit keys, 8 kv heads, 84 us; 204 over 2 of 6400 ..
// 13000, 4 kv heads, with weights 114 to 124 us by the lengths drawn.
#include "walk.cuh"

namespace pa {
namespace walk {
namespace {

constexpr int kTK = 64;
constexpr int kTileBytes = kTK * kD * 2;

__device__ __forceinline__ uint32_t chunk_at(int row, int c) {
    return static_cast<uint32_t>(row * 256 + (c & 1) * 128 + (((c >> 1) ^ (row & 7)) << 4));
}

// Requests tiles of 64 keys.  The 16 rows that a warp's threads load are looked up
// by lanes 0 .. 15, a tile ahead of their use.
template <int ROWS_>  // consecutive rows of a warp, one group of them every 64 / (16 / ROWS_)
struct RowLookup {
    static constexpr int kStride = 4 * ROWS_;  // keys from one group to the next
    int page = kNoPage, slot = 0;
    bool bad = false;
    __device__ __forceinline__ void look(const WalkParams& p, int b, int base, int S) {
        const int lane = threadIdx.x & 31, l = lane & 15;
        const int key = base + ROWS_ * static_cast<int>(threadIdx.x >> 5) + l % ROWS_ + kStride * (l / ROWS_);
        const int lp = key / p.ps;
        slot = key - lp * p.ps;
        page = key < S ? __ldg(p.bt + static_cast<long long>(b) * p.max_npg + lp) : kNoPage;
    }
    __device__ __forceinline__ int rows(const WalkParams& p, int kvh) { return row_in(p, kvh, page, slot, bad); }
};

template <bool Q4>
struct TileLoader;

template <>
struct TileLoader<true> {  // thread: dims 16 grp .. of keys (tid >> 3) + 16 i
    RowLookup<4> rows;
    uint2 c[4][2];
    uint32_t s[4][2];
    __device__ __forceinline__ void request(const WalkParams& p, int kvh, uint32_t, uint32_t) {
        const int lane = threadIdx.x & 31, grp = lane & 7, mine = rows.rows(p, kvh);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long r = __shfl_sync(0xffffffffu, mine, 4 * i + (lane >> 3));
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
    RowLookup<2> rows;
    __device__ __forceinline__ void request(const WalkParams& p, int kvh, uint32_t kbuf, uint32_t vbuf) {
        const int lane = threadIdx.x & 31, c = lane & 15, mine = rows.rows(p, kvh);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = static_cast<int>(threadIdx.x >> 4) + 8 * i;
            const int r = __shfl_sync(0xffffffffu, mine, 2 * i + (lane >> 4));
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
    __shared__ int share[4];
    pdl_launch_dependents();
    if (threadIdx.x == 0) p.split[blockIdx.x] = make_int4(-1, 0, 0, 0);
    zero_bad_rows<F32>(p);
    find_share<ROWS>(p, share);
    const int pos = static_cast<int>(blockIdx.x) * share[1], end = min(pos + share[1], share[0]);
    if (pos >= end) return;
    Segment<ROWS> sg;
    sg.b = share[2];
    sg.S = seq_len(p, sg.b, false);
    sg.at(p, share[3], pos, end);
    const uint32_t buf = smem_u32(smem);
    TileLoader<Q4> ld;
    for (; sg.n > 0; sg.advance(p, end)) {  // segments of the share
    const int b = sg.b, kvh = sg.kvh, S = sg.S;
    const int r0 = sg.rc * ROWS, nrows = min(ROWS, p.R - r0);
    const long long row0 = sg.row0(p);
    int k1, cta_lo;
    sg.bounds(p, k1, cta_lo);
    const int k0 = sg.g0 * kUnit;
    // the last key each of this lane's rows (g, g + 8 of the warp's 16) sees, and
    // the extremes over the warp
    int lim[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int rr = 16 * warp + g + 8 * e;
        lim[e] = rr < nrows ? (p.causal ? (r0 + rr) % p.L + S - p.L : S - 1) : -1;
    }
    int lim_min = min(lim[0] < 0 ? INT_MAX : lim[0], lim[1] < 0 ? INT_MAX : lim[1]), lim_max = max(lim[0], lim[1]);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, o));
        lim_max = max(lim_max, __shfl_xor_sync(0xffffffffu, lim_max, o));
    }
    __syncthreads();  // the buffers of the segment before have been read
    ld.rows.look(p, b, k0, S);
    ld.request(p, kvh, buf, buf + kTileBytes);
    ld.rows.look(p, b, k0 + kTK, S);  // (past the piece: not used)

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

    ld.finish(buf, buf + kTileBytes);
    int cur = 0;
    for (int base = k0; base < k1; base += kTK, cur ^= 1) {
        __syncthreads();  // the tile is whole; the other buffer is no longer read
        const uint32_t kb = buf + cur * 2 * kTileBytes, vb = kb + kTileBytes;
        const uint32_t kn = buf + (cur ^ 1) * 2 * kTileBytes, vn = kn + kTileBytes;
        const bool more = base + kTK < k1;
        if (more) {
            ld.request(p, kvh, kn, vn);
            ld.rows.look(p, b, base + 2 * kTK, S);
        }
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
            // P's A fragments of 16 keys each, then O += P V (fp32: a tile's products on their
            // own, then a rounded add, as the MMA cuts what it adds to)
            uint32_t a[4][4], al[F32 ? 4 : 1][4];
            float ls[2], las[2];  // of this tile: a sum of many small weights keeps them
#pragma unroll
            for (int n = 0; n < 8; ++n)  // keys 8 n .., rows g and g + 8
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float p0 = fast_exp2(fmaf(s[n][2 * e], qs[e], -mu[e]));
                    const float p1 = fast_exp2(fmaf(s[n][2 * e + 1], qs[e], -mu[e]));
                    const int at = 2 * (n & 1) + e;
                    ls[e] = n == 0 ? p0 + p1 : ls[e] + (p0 + p1);
                    if constexpr (Q4) {
                        const uint32_t x = pack_f16x2(p0, p1);
                        a[n >> 1][at] = x;
                        if constexpr (F32) {
                            const float2 f = f16x2_to_float2(x);
                            al[n >> 1][at] = pack_f16x2((p0 - f.x) * kLowScale, (p1 - f.y) * kLowScale);
                        }
                    } else {
                        const uint32_t x = pack_bf16x2(p0, p1);
                        const float2 f = bf16x2_to_float2(x);
                        las[e] = n == 0 ? f.x + f.y : las[e] + (f.x + f.y);
                        a[n >> 1][at] = x;
                    }
                }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[e] += ls[e];
                if constexpr (!Q4) la[e] += las[e];
            }
#pragma unroll
            for (int d = 0; d < 16; d += 2) {  // 16 dims
                float y[2][4], z[2][4];  // V hi, V lo
#pragma unroll
                for (int k = 0; k < 4; ++k) {  // 16 keys
                    uint32_t x[4];
                    ldmatrix_x4_trans(x, vb + chunk_at(16 * k + (lane & 15), d + (lane >> 4)));
                    if constexpr (F32) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (k == 0) {
                                mma_first<Q4>(z[h], al[k], x[2 * h], x[2 * h + 1]);
                                mma_first<Q4>(y[h], a[k], x[2 * h], x[2 * h + 1]);
                            } else {
                                mma<Q4>(z[h], al[k], x[2 * h], x[2 * h + 1]);
                                mma<Q4>(y[h], a[k], x[2 * h], x[2 * h + 1]);
                            }
                        }
                    } else {
                        mma<Q4>(o[d], a[k], x[0], x[1]);
                        mma<Q4>(o[d + 1], a[k], x[2], x[3]);
                    }
                }
                if constexpr (F32) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[d + h][e] += fmaf(z[h][e], kLowStep, y[h][e]);
                }
            }
        }
        if (more) ld.finish(kn, vn);
    }
    // rows g and g + 8: dims 8 d + 2t, + 1
    const bool full = sg.full();
    if (!full && sg.g0 == 0 && threadIdx.x == 0) p.split[blockIdx.x] = sg.crossing(share[1]);
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
        if (full) {
            const long long row = row0 + rr;
            const float inv = at == 0.f ? 0.f : 1.f / at;
#pragma unroll
            for (int d = 0; d < 16; ++d) {
                const float x = o[d][2 * e] * inv, y = o[d][2 * e + 1] * inv;
                if constexpr (F32)
                    *reinterpret_cast<float2*>(static_cast<float*>(p.out) + row * kD + 8 * d + 2 * t) = make_float2(x, y);
                else
                    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + row * kD + 8 * d + 2 * t) = pack_bf16x2(x, y);
            }
            if (t == 0 && p.lse) p.lse[row] = l[e] == 0.f ? __int_as_float(0x7f800000) : m[e] + log2f(l[e]);
        } else {
            const long long row = sg.slot() * ROWS + rr;
            if (t == 0) p.part_ml[row] = make_float4(m[e], at, l[e], 0.f);
            if (l[e] != 0.f) {
#pragma unroll
                for (int d = 0; d < 16; ++d)
                    *reinterpret_cast<float2*>(p.part_o + row * kD + 8 * d + 2 * t) =
                        make_float2(o[d][2 * e], o[d][2 * e + 1]);
            }
        }
    }
    }
    report_pages(p, ld.rows.bad);
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

}  // namespace

pa_status block_attend(const WalkParams& p, const WalkLaunch& w) {
    if (!w.q4) return launch_block<false, false>(p, w.items, w.device, w.stream);
    return w.f32 ? launch_block<true, true>(p, w.items, w.device, w.stream)
                 : launch_block<true, false>(p, w.items, w.device, w.stream);
}

}  // namespace walk
}  // namespace pa
