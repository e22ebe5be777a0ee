// The 8-bit codes of a coded KV cache: e4m3 or int8, one f32 scale per token
// and kv head.
//
//   scale = max(max|x| / qmax, 2^-126),  code = rne(x / scale),  x ~ code * scale
//
// with qmax 448 (e4m3) or 127 (int8).  Codes are widened to f16, which holds
// every code of both types exactly, so that products with them carry no
// rounding of the cache's own.
#pragma once

#include <cuda_fp16.h>

#include "internal.h"

namespace pdattn {

struct Uncoded {};   // a cache of T itself
struct E4m3 {
    static constexpr float kQMax = 448.f;
};
struct Int8 {
    static constexpr float kQMax = 127.f;
};

constexpr float kScaleMin = 1.17549435e-38f;   // 2^-126: a row of zeros keeps a usable scale

// Four codes of one word as two f16 pairs, in order.
template <typename Code>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi);
template <>
__device__ __forceinline__ void widen4<E4m3>(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}
// int8: the byte c + 128 under the exponent of 1024 reads 1024 + 128 + c, an
// integer f16 holds exactly; subtracting 1152 leaves c.
template <>
__device__ __forceinline__ void widen4<Int8>(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
}

// Four values already divided by their scale, with their signs turned -> four
// codes, rounded to nearest even.  (A quotient is past qmax by a rounding at
// most.)
template <typename Code>
__device__ __forceinline__ uint32_t encode4(float2 a, float2 b);
template <>
__device__ __forceinline__ uint32_t encode4<E4m3>(float2 a, float2 b) {
    uint32_t w;
    asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
        " mov.b32 %0, {lo, hi};\n}"
        : "=r"(w) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return w ^ 0x80808080u;
}
// int8: beside 1.5 * 2^23 the last bit is worth 1, so the sum is rounded to an
// integer and its low byte is that integer's.
template <>
__device__ __forceinline__ uint32_t encode4<Int8>(float2 a, float2 b) {
    constexpr float kOnes = 12582912.f;
    const uint32_t lo = __byte_perm(__float_as_uint(__fsub_rn(kOnes, a.x)), __float_as_uint(__fsub_rn(kOnes, a.y)), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(__fsub_rn(kOnes, b.x)), __float_as_uint(__fsub_rn(kOnes, b.y)), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// D = A(16x16 f16, row) * B(16x8 f16, col) + D, fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

__device__ __forceinline__ float lds_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}

}  // namespace pdattn
