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
// merge_kernel joins.  Equal shares keep ragged batches balanced and pay
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
// rounded to f16 (2^-11 relative, and keys below 2^-25 of the row's largest weight are lost:
// less than half a bf16 step while a warp has fewer than 2^17 of them; split in two for
// fp32, 2^-22, with no such limit: kLowScale).  Over bf16 pages the operands are bf16, and
// the row sum that divides O adds the rounded weights.
// Max, sums and O are fp32.  The running max moves only when it grows by more
// than 2^8, so O is rarely rescaled.
//
// Weights: with few rows the scores are left for weights.cu, which adds the rows'
// probabilities in a fixed order (no atomics: a call's results repeat bit for bit).
//
// Measured (G = 4, H_kv = 8, one query position, L2 flushed): 16 sequences of 32768
// 4-bit keys 118 us, 5.1 TB/s of rows read; 64 of 128 .. 4096 45 us, 3.5 TB/s.  No pipe is
// full there (issue 61% of active cycles, ALU 46%): 3.5 warps a scheduler wait for chains of
// a code's conversion, product and exponential; with short contexts 15% is the launch's
// start and end, and a merge follows.  64 of 128 .. 4096 bf16 keys with weights 106 us,
// 5.3 TB/s.
#include "walk.cuh"

namespace pa {
namespace walk {
namespace {

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
    Segment<ROWS> sg;
    int end = 0;  // of this CTA's share
    if (p.whole) {
        int item = static_cast<int>(blockIdx.x);
        sg.rc = item % p.nrc;
        item /= p.nrc;
        sg.kvh = item % p.H_kv;
        sg.b = item / p.H_kv;
        sg.S = seq_len(p, sg.b, sg.rc == 0 && sg.kvh == 0 && threadIdx.x == 0);
        sg.seg = sg.g0 = 0;
        sg.ng = sg.n = (sg.S + kUnit - 1) / kUnit;
    } else {
        if (threadIdx.x == 0) p.split[blockIdx.x] = make_int4(-1, 0, 0, 0);
        zero_bad_rows<F32>(p);
        find_share<ROWS>(p, share);
        const int pos = static_cast<int>(blockIdx.x) * share[1];
        end = min(pos + share[1], share[0]);
        if (pos >= end) return;
        sg.b = share[2];
        sg.S = seq_len(p, sg.b, false);
        sg.at(p, share[3], pos, end);
        if (sg.n == 0) return;
    }
    const uint32_t ring = smem_u32(smem) + warp * 2 * St::kBytes;
    uint32_t st = ring;
    StepWalker<A16, U> wk;
    int pg[2] = {-1, -1};
    QueryFrags<Keys, F32> q[NT];
    // Requests the first stage, the page ids after it and the query rows of `sg`.
    auto open_keys = [&]() {
        int k1, lo;
        sg.bounds(p, k1, lo);
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
        const long long row0 = sg.row0(p);
#pragma unroll
        for (int n = 0; n < NT; ++n) q[n].request(p.q, row0 + 8 * n + g, sg.rc * ROWS + 8 * n + g < p.R, t);
    };
    open_query();
    open_keys();

    for (;;) {  // segments of the share
    const int S = sg.S, b = sg.b, kvh = sg.kvh;
    const int r0 = sg.rc * ROWS, nrows = min(ROWS, p.R - r0);
    const long long row0 = sg.row0(p);
    const int npg = (S + p.ps - 1) / p.ps;
    const int32_t* const table = p.bt + static_cast<long long>(b) * p.max_npg;
    int k1, lim_min;  // last key any row sees + 1 (within the share), last key every row sees
    sg.bounds(p, k1, lim_min);
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
            float ls[2], las[2];  // of this step: a sum of many small weights keeps them
            const float mu[2] = {m[n][0] == neg_inf() ? 0.f : m[n][0], m[n][1] == neg_inf() ? 0.f : m[n][1]};
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) {  // keys g, then g + 8
                    const float p0 = fast_exp2(fmaf(s[n][u][2 * h], qs[n][0], -mu[0]));
                    const float p1 = fast_exp2(fmaf(s[n][u][2 * h + 1], qs[n][1], -mu[1]));
                    const bool first = u == 0 && h == 0;
                    ls[0] = first ? p0 : ls[0] + p0;
                    ls[1] = first ? p1 : ls[1] + p1;
                    if constexpr (F16) {
                        const uint32_t x = pack_f16x2(p0, p1);
                        pb[n][u][h] = movmatrix_trans(x);
                        if constexpr (F32) {
                            const float2 f = f16x2_to_float2(x);
                            pl[n][u][h] = movmatrix_trans(pack_f16x2((p0 - f.x) * kLowScale, (p1 - f.y) * kLowScale));
                        }
                    } else {
                        const uint32_t x = pack_bf16x2(p0, p1);
                        const float2 f = bf16x2_to_float2(x);
                        las[0] = first ? f.x : las[0] + f.x;
                        las[1] = first ? f.y : las[1] + f.y;
                        pb[n][u][h] = movmatrix_trans(x);
                    }
                }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[n][e] += ls[e];
                if constexpr (!F16) la[n][e] += las[e];
            }
        }
        Values vv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) vv[u].load(st, u, g, t);
        if (base + kStep > S) {  // slots past the context may hold anything
#pragma unroll
            for (int u = 0; u < U; ++u) vv[u].cut(S - base - 16 * u, t);
        }
        // O^T += V^T P^T (fp32: each step's products on their own, then a rounded add.  The
        // MMA cuts what it adds to: over thousands of keys that would show, 5e-6 of the
        // result over 3000 against 5e-7.)
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
                        float(&acc)[4] = o[n][4 * i + mm];
                        if constexpr (F32) {
                            float x[4];
                            mma_first<F16>(x, a[mm], pl[n][u][0], pl[n][u][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) x[e] *= kLowStep;
                            mma<F16>(x, a[mm], pb[n][u][0], pb[n][u][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[e] += x[e];
                        } else {
                            mma<F16>(acc, a[mm], pb[n][u][0], pb[n][u][1]);
                        }
                    }
            }
        }
        st = st_next;
    }
    const Segment<ROWS> done = sg;
    bool more = false;
    if (!p.whole) {
        sg.advance(p, end);
        more = sg.n > 0;
    }
    if (more) {
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
    const bool full = done.full();
    if (!full && done.g0 == 0 && threadIdx.x == 0) p.split[blockIdx.x] = done.crossing(share[1]);
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
        const float Mu = M == neg_inf() ? 0.f : M;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float* const mw_ = mr + w * mrows * kMerge;
            const float a = fast_exp2(mv[w] - Mu);  // a warp without keys: 0 times zeros
            const float4 x = *reinterpret_cast<const float4*>(mw_ + 4 * lane);
            acc.x += a * x.x;
            acc.y += a * x.y;
            acc.z += a * x.z;
            acc.w += a * x.w;
            at += a * mw_[kD + 1];
            lt += a * mw_[kD + 2];
        }
        if (full) {
            store_row<F32>(p, row0 + rr, lane, acc, at, lt, M);
        } else {
            const long long row = done.slot() * ROWS + rr;
            if (lane == 0) p.part_ml[row] = make_float4(M, at, lt, 0.f);
            if (lt != 0.f) *reinterpret_cast<float4*>(p.part_o + row * kD + 4 * lane) = acc;
        }
    }
    if (!more) break;
    __syncthreads();  // the merge buffer is free
    }
    cp_async_wait<0>();
    report_pages(p, wk.bad);
}

// Joins the pieces of the segments that cross shares: CTA (c, y) rows N y .. of the
// segment that starts in share c.  Its four warps take every fourth piece, N rows of
// U pieces in flight, four dims a lane.
template <bool F32, int N, int U>
__global__ void __launch_bounds__(kWarps * 32) merge_kernel(const WalkParams p, int rows_cta) {
    __shared__ float4 mls[kWarps][N];
    __shared__ float4 os[kWarps][N][32];
    pdl_launch_dependents();
    pdl_wait_primary();
    const int c = blockIdx.x, r0 = N * static_cast<int>(blockIdx.y);
    const int4 sp = p.split[c];
    if (sp.x < 0 || sp.z * rows_cta + r0 >= p.R) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float4 st[N], acc[N];  // max, sum of the applied weights, sum
#pragma unroll
    for (int i = 0; i < N; ++i) {
        st[i] = make_float4(neg_inf(), 0.f, 0.f, 0.f);
        acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    auto add = [](float4& s, float4& o, const float4 v, const float4 x) {
        if (v.z == 0.f) return;  // no key (and x was not written)
        const float m = fmaxf(s.x, v.x), a = fast_exp2(s.x - m), b = fast_exp2(v.x - m);
        s = make_float4(m, s.y * a + v.y * b, s.z * a + v.z * b, 0.f);
        o = make_float4(o.x * a + x.x * b, o.y * a + x.y * b, o.z * a + x.z * b, o.w * a + x.w * b);
    };
    for (int k0 = c + warp; k0 <= sp.w; k0 += U * kWarps) {
        float4 v[U][N], x[U][N];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u * kWarps;
            const long long row = (2ll * k + (k == c ? 1 : 0)) * rows_cta + r0;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                v[u][i] = make_float4(neg_inf(), 0.f, 0.f, 0.f);
                if (k <= sp.w) {
                    v[u][i] = p.part_ml[row + i];
                    x[u][i] = *reinterpret_cast<const float4*>(p.part_o + (row + i) * kD + 4 * lane);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < N; ++i) add(st[i], acc[i], v[u][i], x[u][i]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (lane == 0) mls[warp][i] = st[i];
        os[warp][i][lane] = acc[i];
    }
    __syncthreads();
    const int rr = sp.z * rows_cta + r0 + warp;  // a warp per row
    if (warp >= N || rr >= p.R) return;
    float4 s = mls[0][warp], o = os[0][warp][lane];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) add(s, o, mls[w][warp], os[w][warp][lane]);
    store_row<F32>(p, (static_cast<long long>(sp.x) * p.H_kv + sp.y) * p.R + rr, lane, o, s.y, s.z, s.x);
}

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

}  // namespace

int walk_resident(int nt, bool q4, bool f32, int rows) {
    // (bf16 pages: 16 KB of stages a warp leave room for three CTAs of 4 merge rows)
    return !q4 && nt == 1 && rows > 4 ? 2 : resident_ctas(nt, q4, f32);
}

pa_status walk_attend(const WalkParams& p, const WalkLaunch& w) {
    if (!w.q4)
        return w.nt == 2 ? launch_walk_for<BfKeys, BfValues, 2, false>(p, w.items, w.device, w.stream)
                         : launch_walk_for<BfKeys, BfValues, 1, false>(p, w.items, w.device, w.stream);
    if (w.f32) return launch_walk_for<Q4Keys, Q4Values, 1, true>(p, w.items, w.device, w.stream);
    return w.nt == 2 ? launch_walk_for<Q4Keys, Q4Values, 2, false>(p, w.items, w.device, w.stream)
                     : launch_walk_for<Q4Keys, Q4Values, 1, false>(p, w.items, w.device, w.stream);
}

pa_status merge_shares(const WalkParams& p, int rows_cta, int shares, bool f32, cudaStream_t stream) {
    // few rows: a CTA per row; block_kernel's 64: four rows a CTA
    const int rows = rows_cta < p.R ? rows_cta : p.R, n = rows_cta <= 16 ? 1 : 4;
    const dim3 grid(static_cast<unsigned>(shares), static_cast<unsigned>((rows + n - 1) / n));
    auto* const kernel = n == 1 ? (f32 ? merge_kernel<true, 1, 4> : merge_kernel<false, 1, 4>)
                                : (f32 ? merge_kernel<true, 4, 1> : merge_kernel<false, 4, 1>);
    return launch_dependent(kernel, grid, kWarps * 32, 0, stream, p, rows_cta) ? PA_OK : PA_ERR_CUDA;
}

}  // namespace walk
}  // namespace pa
