// 8-bit codes (e4m3: sign, 4 exponent bits, 3 mantissa bits, largest value 448)
// and the scale of a quantised row.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace sdv {
namespace {

// two values to two codes, to nearest even, the first in the low byte; beyond 448 gives 448
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n"
        " mov.b32 %0, {l, h};\n}\n" : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}
// and back, exact
__device__ __forceinline__ float2 from_e4m3x2(uint16_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
__device__ __forceinline__ float4 from_e4m3x4(uint32_t codes) {
    const float2 a = from_e4m3x2((uint16_t)codes), b = from_e4m3x2((uint16_t)(codes >> 16));
    return make_float4(a.x, a.y, b.x, b.y);
}

// a row's scale by its largest magnitude m, and its elements u as u 448 / m
constexpr float kE4m3Max = 448.f, kE4m3Tiny = 0x1p-100f;
__device__ __forceinline__ float e4m3_scale(float amax) { return __fdiv_rn(fmaxf(amax, kE4m3Tiny), kE4m3Max); }
// u 448 / m to the nearest fp32 value.  For bf16 rows u 448 / m often is the middle of two codes, and a product
// with 448 / m, rounded before, then falls to either side by chance (1 code in 1,000).  So the product q is
// corrected by what it leaves (Markstein's correction of a quotient): q + (7/8 u - q (m / 512)) (512 / m), which
// cannot overflow, and whose bracket rounds at 2^-28 of u.
struct RowCodes {
    float mul, part, inv;            // 448 / m, m / 512, 512 / m
    __device__ __forceinline__ explicit RowCodes(float amax) {
        const float m = fmaxf(amax, kE4m3Tiny);
        mul = __fdiv_rn(kE4m3Max, m);
        part = m * 0x1p-9f;
        inv = mul * (512.f / 448.f);
    }
    __device__ __forceinline__ float operator()(float u) const {
        const float q = __fmul_rn(u, mul);
        return fmaf(fmaf(u, -0.125f, fmaf(-q, part, u)), inv, q);
    }
    __device__ __forceinline__ float2 operator()(float2 u) const {
        const float2 q = __fmul2_rn(u, make_float2(mul, mul));
        const float2 left = __ffma2_rn(u, make_float2(-0.125f, -0.125f),
                                       __ffma2_rn(make_float2(-q.x, -q.y), make_float2(part, part), u));
        return __ffma2_rn(left, make_float2(inv, inv), q);
    }
};

}  // namespace

// storage of a code
struct E4m3 { uint8_t c; };
template <> struct Elem<E4m3> {
    static constexpr int kPerVec = 8;   // an 8-byte load
    __device__ __forceinline__ static void load_vec(const E4m3 *p, float (&f)[8]) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
        const float4 a = from_e4m3x4(v.x), b = from_e4m3x4(v.y);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
};

}  // namespace sdv
