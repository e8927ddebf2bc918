// fp4.cuh -- conversions of the 4-bit cache: E2M1 codes and E4M3 scales.
//
// All four conversions are single instructions on sm_103a at 64 lanes per
// clock and SM (measured), so two E2M1 codes become two fp16 values for the
// price of one logic operation.  value(c) * value(s) has at most 6
// significant bits and lies in [2^-10, 2688]: exact in fp16.
#pragma once

#include "pa_device.cuh"

namespace pa {

// Byte i of w as two E2M1 codes -> fp16x2 (low four bits in the low half).
template <int I>
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t w) {
    uint32_t d;
    if constexpr (I == 0)
        asm("{\n\t.reg .b8 a, b, c, e;\n\tmov.b32 {a, b, c, e}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(d) : "r"(w));
    else if constexpr (I == 1)
        asm("{\n\t.reg .b8 a, b, c, e;\n\tmov.b32 {a, b, c, e}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(d) : "r"(w));
    else if constexpr (I == 2)
        asm("{\n\t.reg .b8 a, b, c, e;\n\tmov.b32 {a, b, c, e}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(d) : "r"(w));
    else
        asm("{\n\t.reg .b8 a, b, c, e;\n\tmov.b32 {a, b, c, e}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, e;\n\t}" : "=r"(d) : "r"(w));
    return d;
}

// Two E4M3 bytes -> fp16x2 (low byte in the low half).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)two));
    return d;
}

// Nearest E4M3 byte of x >= 0, ties to even, saturating at 448.
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(0.f), "f"(x));
    return d & 0xffu;
}

// Nearest E2M1 codes of (lo, hi), ties to even, saturating at 6: one byte.
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2(float lo, float hi) {
    uint32_t d;
    asm("{\n\t.reg .b8 a;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %1, %2;\n\tcvt.u32.u8 %0, a;\n\t}" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// 8 consecutive elements: fp32 in, T out.
__device__ __forceinline__ void load8(const float *src, float (&x)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(src), b = *(reinterpret_cast<const float4 *>(src) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
template <typename T>
__device__ __forceinline__ void store8(T *dst, const float (&x)[8]) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4 *>(dst) = make_float4(x[0], x[1], x[2], x[3]);
        *(reinterpret_cast<float4 *>(dst) + 1) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint4 a;
        a.x = Elem<T>::pack2(x[0], x[1]);
        a.y = Elem<T>::pack2(x[2], x[3]);
        a.z = Elem<T>::pack2(x[4], x[5]);
        a.w = Elem<T>::pack2(x[6], x[7]);
        *reinterpret_cast<uint4 *>(dst) = a;
    }
}

}  // namespace pa
