// q4.cuh -- device helpers of the 4-bit row format.
//
// A row is 128 values: 64 bytes of e2m1 codes (dim 2i in the low half of byte
// i, dim 2i + 1 in the high half) and 8 e4m3 scales, one per 16 dims; a value
// is code * scale.  A code has 2 significant bits and a scale 4, so a product
// has at most 6 and lies in [2^-10, 2688]: exact in f16, bf16 and fp32.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace pa {

// The two e2m1 codes of the low byte of b as f16x2 (low half = low code).
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t b) {
    uint32_t r;
    asm("{\n\t.reg .b8 c;\n\tmov.b32 {c, _, _, _}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}"
        : "=r"(r)
        : "r"(b));
    return r;
}

// The eight codes of a word as four f16x2: v[i] = the codes of byte i.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&v)[4]) {
    asm("{\n\t.reg .b8 c0, c1, c2, c3;\n\tmov.b32 {c0, c1, c2, c3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, c0;\n\tcvt.rn.f16x2.e2m1x2 %1, c1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c2;\n\tcvt.rn.f16x2.e2m1x2 %3, c3;\n\t}"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
        : "r"(w));
}

// Two e4m3 scales (low 16 bits) as f16x2.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t b) {
    uint32_t r;
    asm("{\n\t.reg .b16 s;\n\tcvt.u16.u32 s, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, s;\n\t}"
        : "=r"(r)
        : "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t w) {
    float2 r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\t"
        "cvt.f32.f16 %1, h;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(w));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// D += A B with f16 or bf16 operands (fragment layouts as mma_16816 in ptx.cuh;
// not volatile, so that the compiler may move the products between the
// conversions that feed them).
__device__ __forceinline__ void mma_16816_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_16816_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// D = A B.
__device__ __forceinline__ void mma_16816_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_16816_bf16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                                     uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

template <bool F16>
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        mma_16816_f16_first(d, a, b0, b1);
    else
        mma_16816_bf16_first(d, a, b0, b1);
}
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        mma_16816_f16(d, a, b0, b1);
    else
        mma_16816_bf16(d, a, b0, b1);
}

// The power of two that takes a row with largest magnitude mx into f16's range
// (mx into [2^14, 2^15)), and its inverse.  Rows with an inf or NaN stay as they
// are; the exponent is cut so that both factors are normal numbers.
__device__ __forceinline__ void f16_scale(float mx, float& up, float& down) {
    const int e = static_cast<int>(__float_as_uint(mx) >> 23) - 127;  // -127: zero or subnormal
    const int k = e >= 128 ? 0 : min(14 - e, 126);
    up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
    down = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
}

}  // namespace pa
