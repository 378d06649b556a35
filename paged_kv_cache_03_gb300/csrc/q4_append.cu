// q4_append.cu -- new K/V rows rounded to 4 bits into their pages, and the
// dense read-back of such pages.
//
// A group of 16 dims gets the scale s = RNE_e4m3(max|x| / 6), kept in [2^-9,
// 448], and the codes RNE_e2m1(x / s), which saturate at +-6.  Both divisions
// are fp32: a quotient that rounds to a border between two codes (at most 3
// significant bits) or two scales (5 bits) is exactly on it, because x and
// border * s are both fp32 numbers, and two different ones lie more than half
// an ulp of the quotient apart; so every code is the one of the real quotient.
// A NaN in a group makes its scale NaN.
//
// The new tokens of sequence b are its last L positions, through the block
// table as in append.cu; sequences or pages that break the contract set the
// same flags and are skipped.
#include <climits>

#include "cache.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace pa {
namespace {

struct Q4AppendParams {
    const void* k_new;
    const void* v_new;
    pa_q4_pool pool;
    const int32_t* bt;
    const int32_t* ctx;
    uint32_t* flag;
    int rows;  // B * H_kv * L new rows (host-checked: 8 threads a row fit an int)
    int H_kv, L, ps, max_npg, num_pages;
    long long max_S;
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// e4m3 byte of x >= 0, round to nearest even, saturating at 448 (NaN: 0x7f).
__device__ __forceinline__ uint32_t float_to_e4m3(float x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return r & 0xffu;
}

// e2m1 codes of (lo, hi): low and high half of a byte.
__device__ __forceinline__ uint32_t float_to_e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %2, %1;\n\t"
        "mov.b32 %0, {c, 0, 0, 0};\n\t}"
        : "=r"(r)
        : "f"(lo), "f"(hi));
    return r;
}

// 16 consecutive values of a row.
template <typename T>
__device__ __forceinline__ void load16(const T* src, float (&x)[16]) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 w = __ldcs(reinterpret_cast<const uint4*>(src) + i);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = bf16x2_to_float2(ww[j]);
                x[8 * i + 2 * j] = f.x;
                x[8 * i + 2 * j + 1] = f.y;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 f = __ldcs(reinterpret_cast<const float4*>(src) + i);
            x[4 * i] = f.x;
            x[4 * i + 1] = f.y;
            x[4 * i + 2] = f.z;
            x[4 * i + 3] = f.w;
        }
    }
}

// The scale byte and the codes of 16 values.  x / s is rounded correctly by
// Markstein's correction: with r the correctly rounded 1 / s and q0 = x r, the
// remainder x - q0 s is exact in one FMA and q0 + r (x - q0 s) rounds to the
// quotient.  |x| is cut to 8 s first (its code stays 6), so nothing overflows.
__device__ __forceinline__ uint2 encode16(const float (&x)[16], uint32_t& sb) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = max_nan(amax, fabsf(x[i]));
    sb = float_to_e4m3(max_nan(__fdiv_rn(amax, 6.f), 0.001953125f));
    const float sc = f16x2_to_float2(e4m3x2_to_f16x2(sb)).x;
    const float r = __frcp_rn(sc), cut = 8.f * sc;
    uint32_t code[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float y[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float c = fminf(fmaxf(x[2 * i + e], -cut), cut);
            const float q0 = c * r;
            y[e] = copysignf(fmaf(fmaf(-q0, sc, c), r, q0), c);  // (-0 stays -0)
        }
        code[i >> 2] |= float_to_e2m1x2(y[0], y[1]) << (8 * (i & 3));
    }
    return make_uint2(code[0], code[1]);
}

// Eight threads a row, 16 dims each, its key and its value: 512 bytes in (bf16) for 144
// out.  4 x 8 heads x 2048 rows 15.8 us, 3.0 TB/s.  Bound by latency: 8.3 M warp instructions
// are about 7 us of issue, and a thread loads its row, then encodes it, with no other row
// on its way.
template <typename T>
__global__ void __launch_bounds__(256) q4_append_kernel(const Q4AppendParams p) {
    const int u = static_cast<int>(blockIdx.x * blockDim.x + threadIdx.x);
    const int row = u >> 3, grp = u & 7;
    if (row >= p.rows) return;
    const int bk = row / p.L, t = row - bk * p.L;
    const int b = bk / p.H_kv, kvh = bk - b * p.H_kv;
    const int S = __ldg(p.ctx + b);
    if (S < p.L || static_cast<long long>(S) > p.max_S) {
        if (kvh == 0 && t == 0 && grp == 0) atomicOr(p.flag, PA_FLAG_BAD_CONTEXT);
        return;
    }
    const int s = S - p.L + t;
    const int lp = s / p.ps, slot = s - lp * p.ps;
    const int pp = __ldg(p.bt + static_cast<long long>(b) * p.max_npg + lp);
    const long long src = static_cast<long long>(row) * kHeadDim + grp * 16;
    float x[2][16];
    load16(static_cast<const T*>(p.k_new) + src, x[0]);
    load16(static_cast<const T*>(p.v_new) + src, x[1]);
    if (pp < 0 || pp >= p.num_pages) {
        if (grp == 0) atomicOr(p.flag, PA_FLAG_BAD_PAGE);
        return;
    }
    const long long dst = (static_cast<long long>(pp) * p.H_kv + kvh) * p.ps + slot;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        uint32_t sb;
        const uint2 code = encode16(x[kv], sb);
        uint8_t* const codes = static_cast<uint8_t*>(kv ? p.pool.value_codes : p.pool.key_codes);
        uint8_t* const scales = static_cast<uint8_t*>(kv ? p.pool.value_scales : p.pool.key_scales);
        *reinterpret_cast<uint2*>(codes + dst * kQ4CodeBytes + grp * 8) = code;
        scales[dst * kQ4Groups + grp] = static_cast<uint8_t>(sb);
    }
}

struct Q4GatherParams {
    pa_q4_pool pool;
    const int32_t* bt;
    const int32_t* ctx;
    void* k;
    void* v;
    uint32_t* flag;
    int H_kv, n, tail, ps, max_npg, num_pages, ntile;
    int fill;     // rows outside [0, context_lens[b]): 1 zeros, 0 not written
    int32_t* id;  // if not null: id[b] = b, id[nid + b] = the length (0 for a bad one)
    int nid;
    long long max_S;
};

constexpr int kGatherRows = 64;

// A block takes 64 dense rows of one (sequence, kv head), keys and values: 8
// lanes a row, each 8 code bytes and a scale in, 16 values out.  Bound by the
// rows it writes (256 bytes in bf16 for 72 read): 32 x 8 x 1024 rows 27 us, 5.9 TB/s.
template <typename T>
__global__ void __launch_bounds__(256) q4_gather_kernel(const Q4GatherParams p) {
    const int tile = static_cast<int>(blockIdx.x) % p.ntile, bk = static_cast<int>(blockIdx.x) / p.ntile;
    const int b = bk / p.H_kv, kvh = bk - b * p.H_kv;
    const int grp = threadIdx.x & 7;
    int S = __ldg(p.ctx + b);
    if (S < 0 || static_cast<long long>(S) > p.max_S) {
        if (kvh == 0 && tile == 0 && threadIdx.x == 0) atomicOr(p.flag, PA_FLAG_BAD_CONTEXT);
        S = 0;
    }
    if (p.id && kvh == 0 && tile == 0 && threadIdx.x == 0) {
        p.id[b] = b;
        p.id[p.nid + b] = S;
    }
    if (!p.fill && tile * kGatherRows >= S) return;
    uint2 code[2][2];
    uint32_t sb[2][2];
    bool write[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = tile * kGatherRows + 32 * e + static_cast<int>(threadIdx.x >> 3);
        const long long s = p.tail ? static_cast<long long>(S) - p.n + i : i;
        const bool in = s >= 0 && s < S;
        write[e] = i < p.n && (in || p.fill);
        code[e][0] = code[e][1] = make_uint2(0u, 0u);
        sb[e][0] = sb[e][1] = 0u;
        if (i < p.n && in) {
            const int lp = static_cast<int>(s) / p.ps, slot = static_cast<int>(s) - lp * p.ps;
            const int pp = __ldg(p.bt + static_cast<long long>(b) * p.max_npg + lp);
            if (pp >= 0 && pp < p.num_pages) {
                const long long src = (static_cast<long long>(pp) * p.H_kv + kvh) * p.ps + slot;
                const uint8_t* const kc = static_cast<const uint8_t*>(p.pool.key_codes);
                const uint8_t* const vc = static_cast<const uint8_t*>(p.pool.value_codes);
                code[e][0] = *reinterpret_cast<const uint2*>(kc + src * kQ4CodeBytes + grp * 8);
                code[e][1] = *reinterpret_cast<const uint2*>(vc + src * kQ4CodeBytes + grp * 8);
                sb[e][0] = static_cast<const uint8_t*>(p.pool.key_scales)[src * kQ4Groups + grp];
                sb[e][1] = static_cast<const uint8_t*>(p.pool.value_scales)[src * kQ4Groups + grp];
            } else if (grp == 0) {
                atomicOr(p.flag, PA_FLAG_BAD_PAGE);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (!write[e]) continue;
        const long long row = static_cast<long long>(bk) * p.n + tile * kGatherRows + 32 * e + (threadIdx.x >> 3);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint32_t s2 = e4m3x2_to_f16x2(sb[e][kv] | (sb[e][kv] << 8));
            uint32_t h[8];
            e2m1x8_to_f16x2(code[e][kv].x, *reinterpret_cast<uint32_t(*)[4]>(h));
            e2m1x8_to_f16x2(code[e][kv].y, *reinterpret_cast<uint32_t(*)[4]>(h + 4));
            T* const dst = static_cast<T*>(kv ? p.v : p.k) + row * kHeadDim + grp * 16;
            float2 f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = f16x2_to_float2(hmul2(h[j], s2));
            if constexpr (sizeof(T) == 2) {
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = pack_bf16x2(f[j].x, f[j].y);
                // 32 bytes a lane where the caller's buffer allows them
                if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
                    st_global_v8(dst, w);
                } else {
                    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    reinterpret_cast<float4*>(dst)[j] =
                        make_float4(f[2 * j].x, f[2 * j].y, f[2 * j + 1].x, f[2 * j + 1].y);
            }
        }
    }
}

}  // namespace

pa_status q4_append_launch(const pa_shape& sh, const void* k_new, const void* v_new,
                           const pa_q4_pool& pool, const int32_t* bt, const int32_t* ctx,
                           uint32_t* flag, cudaStream_t stream) {
    Q4AppendParams p;
    p.k_new = k_new;
    p.v_new = v_new;
    p.pool = pool;
    p.bt = bt;
    p.ctx = ctx;
    p.flag = flag;
    const long long rows = static_cast<long long>(sh.B) * sh.H_kv * sh.L;
    if (rows * 8 > INT_MAX - 256) return PA_ERR_UNSUPPORTED;
    p.rows = static_cast<int>(rows);
    p.H_kv = sh.H_kv;
    p.L = sh.L;
    p.ps = sh.page_size;
    p.max_npg = sh.max_pages_per_seq;
    p.num_pages = sh.num_pages;
    p.max_S = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    const unsigned grid = static_cast<unsigned>((rows * 8 + 255) / 256);
    if (sh.dtype == PA_BF16)
        q4_append_kernel<uint16_t><<<grid, 256, 0, stream>>>(p);
    else
        q4_append_kernel<float><<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status q4_gather_launch(const pa_shape& sh, const pa_q4_pool& pool, const int32_t* bt,
                           const int32_t* ctx, int n, int tail, int fill, int32_t* id, int nid,
                           void* k_dense, void* v_dense, uint32_t* flag, cudaStream_t stream) {
    Q4GatherParams p;
    p.pool = pool;
    p.bt = bt;
    p.ctx = ctx;
    p.k = k_dense;
    p.v = v_dense;
    p.flag = flag;
    p.H_kv = sh.H_kv;
    p.n = n;
    p.tail = tail;
    p.fill = fill;
    p.id = id;
    p.nid = nid;
    p.ps = sh.page_size;
    p.max_npg = sh.max_pages_per_seq;
    p.num_pages = sh.num_pages;
    p.ntile = (n + kGatherRows - 1) / kGatherRows;
    p.max_S = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    const long long blocks = static_cast<long long>(sh.B) * sh.H_kv * p.ntile;
    if (blocks > INT_MAX || n > INT_MAX - kGatherRows) return PA_ERR_UNSUPPORTED;
    if (sh.dtype == PA_BF16)
        q4_gather_kernel<uint16_t><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(p);
    else
        q4_gather_kernel<float><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
