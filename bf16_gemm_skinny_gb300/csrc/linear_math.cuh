// linear_math.cuh -- activations, their derivatives and the 16-bit types of the
// feed-forward layer kernels.
//
//   silu       z s(z),                     s(v) = 1 / (1 + e^-v)
//   gelu       z Phi(z),                   Phi the normal distribution function
//   gelu_tanh  z s(2c (z + a z^3)),        c = sqrt(2/pi), a = 0.044715: the usual
//              z/2 (1 + tanh(c (z + a z^3))) by (1 + tanh v)/2 = s(2v), which does
//              not cancel where tanh nears -1
//   derivatives: s (1 + z (1-s));  Phi + z phi;  s + z s (1-s) 2c (1 + 3 a z^2)
// All in FP32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "linear_internal.h"

namespace bsk {
namespace {

template <int TYPE>
__device__ __forceinline__ float to_f32(uint16_t b)
{
    if constexpr (TYPE == kTypeBF16) return __uint_as_float(static_cast<uint32_t>(b) << 16);
    else return __half2float(__ushort_as_half(b));
}
template <int TYPE>
__device__ __forceinline__ uint16_t to_16(float v)
{
    if constexpr (TYPE == kTypeBF16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    else return __half_as_ushort(__float2half_rn(v));
}
// Two values of a 32-bit word (element 0 in the low half), and back (one rounding each).
template <int TYPE>
__device__ __forceinline__ float2 unpack2(uint32_t w)
{
    if constexpr (TYPE == kTypeBF16) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    } else {
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    }
}
template <int TYPE>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if constexpr (TYPE == kTypeBF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}

__device__ __forceinline__ float sigmoid_f(float v)
{
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + __expf(-v)));
    return r;
}

constexpr float kGeluC2 = 1.5957691216057308f;   // 2 sqrt(2/pi)
constexpr float kGeluA = 0.044715f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

template <int ACT>
__device__ __forceinline__ float act_value(float z)
{
    if constexpr (ACT == kActRelu) return z <= 0.f ? 0.f : z;   // a NaN stays
    else if constexpr (ACT == kActSilu) return z * sigmoid_f(z);
    else if constexpr (ACT == kActGelu) return z * normcdff(z);
    else if constexpr (ACT == kActGeluTanh) return z * sigmoid_f(kGeluC2 * (z + kGeluA * z * z * z));
    else return z;
}

// act(z) and act'(z).
template <int ACT>
__device__ __forceinline__ float2 act_value_slope(float z)
{
    if constexpr (ACT == kActRelu) {
        return make_float2(z <= 0.f ? 0.f : z, z <= 0.f ? 0.f : (z == z ? 1.f : z));
    } else if constexpr (ACT == kActSilu) {
        const float s = sigmoid_f(z);
        return make_float2(z * s, s * (1.f + z * (1.f - s)));
    } else if constexpr (ACT == kActGelu) {
        const float p = normcdff(z);
        return make_float2(z * p, p + z * kInvSqrt2Pi * __expf(-0.5f * z * z));
    } else if constexpr (ACT == kActGeluTanh) {
        const float s = sigmoid_f(kGeluC2 * (z + kGeluA * z * z * z));
        // beyond 16 s is 0 or 1 and the second term 0; the clamp keeps 0 * infinity out of it
        const float c = fminf(fmaxf(z, -16.f), 16.f);
        return make_float2(z * s, s + c * s * (1.f - s) * (kGeluC2 * (1.f + 3.f * kGeluA * c * c)));
    } else {
        return make_float2(z, 1.f);
    }
}

}  // namespace
}  // namespace bsk
