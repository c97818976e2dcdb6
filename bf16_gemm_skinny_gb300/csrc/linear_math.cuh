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

// 2^x, and 1/x, by the hardware's approximations (2 units in the last place and 1).
__device__ __forceinline__ float exp2_f(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_f(float x)
{
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// d[i] = 1 / d[i] of N values from 1 to 2^30.  The special-function units give 16 results a
// clock and SM, and e^v and 1/x of every value keep them busy longer than HBM takes for the values
// (6992 x 8512 outputs: 27 us): for four values one reciprocal of their product and nine multiplications.
// A value's last bits so depend on the three beside it, and on nothing else.
template <int N>
__device__ __forceinline__ void rcp_all(float (&d)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float ab = d[i] * d[i + 1], cd = d[i + 2] * d[i + 3];
        const float x = rcp_f(ab * cd);
        const float rab = x * cd, rcd = x * ab;
        const float a = rab * d[i + 1], c = rcd * d[i + 3];
        d[i + 1] = rab * d[i];
        d[i] = a;
        d[i + 3] = rcd * d[i + 2];
        d[i + 2] = c;
    }
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluC2 = 1.5957691216057308f;   // 2 sqrt(2/pi)
constexpr float kGeluA = 0.044715f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// The lower tail of the normal distribution, Phi(-|z|) = t Q(t) e^(-z^2 / 2) with t =
// 1 / (1 + 0.4 |z| / sqrt 2): Q is a polynomial fitted here to erfc(x) e^(x^2) / (2t), x = |z| / sqrt 2, for all t in
// (0, 1], largest relative error 1.3e-7 (the form of Press et al., Numerical Recipes, section 6.2:
// a tail keeps its relative accuracy, where 1 + erf would cancel).
__device__ __forceinline__ float normal_tail(float t, float e)
{
    float q = 0.025129861f;
    q = fmaf(q, t, -0.091446319f);
    q = fmaf(q, t, 0.084536198f);
    q = fmaf(q, t, -0.0027988206f);
    q = fmaf(q, t, 0.070713668f);
    q = fmaf(q, t, 0.084271442f);
    q = fmaf(q, t, 0.1039213f);
    q = fmaf(q, t, 0.11283480f);
    q = fmaf(q, t, 0.11283793f);
    return q * t * e;
}

// act(z) of N values (a multiple of 4), in place; SLOPE: act'(z) beside it.
template <int ACT, bool SLOPE, int N>
__device__ __forceinline__ void act_values(float (&z)[N], float (&slope)[N])
{
    static_assert(N % 4 == 0, "reciprocals go by four");
    if constexpr (ACT == kActNone) {
        if constexpr (SLOPE) {
#pragma unroll
            for (int i = 0; i < N; ++i) slope[i] = 1.f;
        }
    } else if constexpr (ACT == kActRelu) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (SLOPE) slope[i] = z[i] <= 0.f ? 0.f : (z[i] == z[i] ? 1.f : z[i]);
            z[i] = z[i] <= 0.f ? 0.f : z[i];   // a NaN stays
        }
    } else {
        // s(v) = 1 / (1 + 2^a), a = -v log2(e); above kFar the 1 counts for nothing, and s is 2^-a =
        // 1 / (1 + 2^kFar) 2^(kFar - a): no factor of a product passes 2^30
        constexpr float kFar = 30.f;
        float r[N], e[N];
        bool far = false;
        auto minus_v = [](float x) {
            return ACT == kActSilu ? x * -kLog2e : x * fmaf(-kLog2e * kGeluC2 * kGeluA * x, x, -kLog2e * kGeluC2);
        };
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (ACT == kActGelu) {
                e[i] = exp2_f(z[i] * z[i] * (-0.5f * kLog2e));
                r[i] = fmaf(fminf(fabsf(z[i]), 1e6f), 0.28284271247461901f, 1.f);
            } else {
                const float a = minus_v(z[i]);
                far = far || a > kFar;
                r[i] = 1.f + exp2_f(fminf(a, kFar));
            }
        }
        rcp_all<N>(r);
        if (ACT != kActGelu && far) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float a = minus_v(z[i]);
                if (a > kFar) r[i] *= exp2_f(kFar - a);
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (ACT == kActGelu) {
                const float tail = normal_tail(r[i], e[i]);
                const float phi = z[i] <= 0.f ? tail : 1.f - tail;
                if constexpr (SLOPE) slope[i] = fmaf(z[i] * kInvSqrt2Pi, e[i], phi);
                z[i] *= phi;
            } else {
                const float s = r[i];
                if constexpr (SLOPE && ACT == kActSilu) slope[i] = s * fmaf(z[i], 1.f - s, 1.f);
                if constexpr (SLOPE && ACT == kActGeluTanh) {
                    // beyond 16 s is 0 or 1 and the second term 0; the clamp keeps 0 * infinity out of it (and a
                    // NaN in, which fminf would take away)
                    const float c = z[i] > 16.f ? 16.f : z[i] < -16.f ? -16.f : z[i];
                    slope[i] = fmaf(c * s * (1.f - s), fmaf(3.f * kGeluC2 * kGeluA * c, c, kGeluC2), s);
                }
                z[i] *= s;
            }
        }
    }
}

}  // namespace
}  // namespace bsk
