// stage.cuh -- asynchronous copies, and tiles of 128 rows in shared memory in the
// 128-byte swizzle that tcgen05.mma reads: 4-bit rows dequantised on the way, bf16
// rows as they are.
#pragma once
#include "cache.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace pa {

constexpr int kRawStage = 32 * (kQ4CodeBytes + kQ4Groups);  // bytes of 32 4-bit rows
constexpr int kStageHalf = 128 * 128;  // bytes of 128 rows x 64 dims, one swizzled column block

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(ok ? 8 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 16-byte chunk c (of 8) of row r in a 64-dim half, 128-byte swizzle.
__device__ __forceinline__ uint32_t sw128(int r, int c) { return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4)); }

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// 16 bytes and a 16-bit word, or zeros.  Volatile: the requests stay where they
// are issued, a tile before their use, whatever the register pressure.
__device__ __forceinline__ void ldg_or_zero(const void* a, const void* b, bool ok, uint4& x, uint32_t& y) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b16 h;\n\tsetp.ne.b32 p, %7, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\tmov.b16 h, 0;\n\t"
        "@p ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%5];\n\t@p ld.global.nc.b16 h, [%6];\n\t"
        "cvt.u32.u16 %4, h;\n\t}"
        : "=&r"(x.x), "=&r"(x.y), "=&r"(x.z), "=&r"(x.w), "=&r"(y)
        : "l"(a), "l"(b), "r"(static_cast<int>(ok)));
}

// A thread's part of one operand's tile: 32 dims (16 code bytes and two
// scales) of four rows.  Lane bits: 0 and 3 the 32-dim quarter (bit 3 its 64-dim
// half), 1, 2 and 4 the row; row i of warp w is 32 i + 8 w + the lane's.  So eight
// neighbouring lanes store to eight different chunk positions (no bank conflict),
// and a warp reads whole code rows.  Stored as f16 or bf16, both exact.
struct RawTile {
    uint4 c[4];
    uint32_t s[4];
    __device__ static int row_of(int lane) { return ((lane >> 1) & 3) | ((lane >> 4) << 2); }
    __device__ static int quarter(int lane) { return (lane & 1) | ((lane >> 2) & 2); }
    // rows: lane 8 i + r holds the pool row of row 32 i + 8 w + r, -1: zeros
    __device__ __forceinline__ void request(const uint8_t* codes, const uint8_t* scales, int rows, int lane) {
        const int q = quarter(lane), rl = row_of(lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = __shfl_sync(0xffffffffu, rows, 8 * i + rl);
            ldg_or_zero(codes + static_cast<long long>(row) * kQ4CodeBytes + 16 * q,
                        scales + static_cast<long long>(row) * kQ4Groups + 2 * q, row >= 0, c[i], s[i]);
        }
    }
    // The same by way of a warp's kRawStage bytes of shared memory (copy; the caller
    // commits, waits and synchronises the warp; read).
    __device__ __forceinline__ static void copy(uint32_t stage, const uint8_t* codes, const uint8_t* scales, int rows,
                                                int lane) {
        const int q = quarter(lane), rl = row_of(lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = __shfl_sync(0xffffffffu, rows, 8 * i + rl);
            cp_async16(stage + 512 * i + 16 * lane,
                       codes + (row < 0 ? 0 : static_cast<long long>(row) * kQ4CodeBytes) + 16 * q, row >= 0);
        }
        cp_async8(stage + 2048 + 8 * lane, scales + (rows < 0 ? 0 : static_cast<long long>(rows) * kQ4Groups), rows >= 0);
    }
    __device__ __forceinline__ void read(uint32_t stage, int lane) {
        const uint32_t at = stage + 2048 + 8 * row_of(lane) + 2 * quarter(lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(c[i].x), "=r"(c[i].y), "=r"(c[i].z), "=r"(c[i].w)
                         : "r"(stage + 512 * i + 16 * lane));
            uint16_t h;
            asm volatile("ld.shared.b16 %0, [%1];" : "=h"(h) : "r"(at + 64 * i));
            s[i] = h;
        }
    }
    template <bool BF16>
    __device__ __forceinline__ void store(uint32_t tile, int warp, int lane) const {
        const int q = quarter(lane), rl = row_of(lane);
        const uint32_t base = tile + (q >> 1) * kStageHalf + (8 * warp + rl) * 128;
        const uint32_t x0 = ((4 * (q & 1)) ^ rl) << 4;  // chunk 4 (q & 1) + j sits at x0 ^ (j << 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
            const uint32_t s2 = e4m3x2_to_f16x2(s[i]);
            const uint32_t sc[2] = {__byte_perm(s2, s2, 0x1010), __byte_perm(s2, s2, 0x3232)};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t v[4];
                e2m1x8_to_f16x2(w[j], v);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[k] = hmul2(v[k], sc[j >> 1]);
                    if constexpr (BF16) {
                        const float2 f = f16x2_to_float2(v[k]);
                        v[k] = pack_bf16x2(f.x, f.y);
                    }
                }
                sts128(base + (x0 ^ (j << 4)) + i * 4096, v[0], v[1], v[2], v[3]);
            }
        }
    }
};

// The same part of a bf16 tile, 32 rows a warp: two rows at a time, 16 lanes a row.
// The caller commits the copies.
__device__ __forceinline__ void copy_tile(uint32_t tile, const uint8_t* pool, int rows, int warp, int lane) {
    const int c = lane & 15;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int x = 2 * i + (lane >> 4), row = __shfl_sync(0xffffffffu, rows, x);
        cp_async16(tile + (c >> 3) * kStageHalf + sw128(32 * (x >> 3) + 8 * warp + (x & 7), c & 7),
                   pool + (row < 0 ? 0 : static_cast<long long>(row) * (2 * kHeadDim)) + 16 * c, row >= 0);
    }
}

}  // namespace pa
