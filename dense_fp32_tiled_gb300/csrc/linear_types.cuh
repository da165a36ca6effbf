// linear_types.cuh -- element types and activations of the layer operators.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "linear.h"

namespace lt {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f<__half>(float v) {
    return __float2half_rn(v);
}

// Two values in one register, the first in the low half.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t u);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t u) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}

// x = a + b + c to 2^-27 |x|, a and b rounded to nearest; a is cut instead
// where rounding would overflow, and carries an infinity or NaN alone.
__device__ __forceinline__ void pieces(float x, __nv_bfloat16 &a, __nv_bfloat16 &b, __nv_bfloat16 &c) {
    a = __float2bfloat16_rn(x);
    const bool finite = fabsf(x) <= 3.402823466e38f;
    if (finite && fabsf(__bfloat162float(a)) > 3.402823466e38f) a = __float2bfloat16_rz(x);
    const float r = finite ? x - __bfloat162float(a) : 0.0f;
    b = __float2bfloat16_rn(r);
    c = __float2bfloat16_rn(r - __bfloat162float(b));
}

inline int type_bytes(int type) { return type == LINEAR_F32 ? 4 : 2; }

// EXACT (FP32 tensors): the library's exponential and division.  The 16-bit
// types round to 8 or 11 bits afterwards, so there the hardware's approximate
// instructions do, 2^-22 of the value, in the form that takes subnormal numbers
// for 0 (the other one, which __expf and __fdividef compile to, scales around
// them and costs an epilogue of a tile about as much again).
__device__ __forceinline__ float fast_exp2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float fast_reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2E = 1.4426950408889634f;
template <bool EXACT>
__device__ __forceinline__ float logistic(float x) {
    return EXACT ? 1.0f / (1.0f + expf(-x)) : fast_reciprocal(1.0f + fast_exp2(-kLog2E * x));
}
// p = logistic(x), and p (1 - p) without the difference, which for large x is as
// coarse as p: gelu_tanh's slope multiplies it by up to 35 before it vanishes.
template <bool EXACT>
__device__ __forceinline__ float logistic(float x, float &pq) {
    const float e = EXACT ? expf(-fabsf(x)) : fast_exp2(-kLog2E * fabsf(x));
    const float s = EXACT ? 1.0f / (1.0f + e) : fast_reciprocal(1.0f + e);
    pq = e * s * s;
    return x < 0.0f ? e * s : s;
}
constexpr float kGeluA = 1.5957691216057308f;   // 2 sqrt(2/pi): (1 + tanh u) / 2 = logistic(2 u)
constexpr float kGeluB = 0.044715f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// The normal distribution's upper tail at |z|, erfc(|z| / sqrt 2) / 2, and
// exp(-z^2 / 2) on the way, for the 16-bit types: exp(-z^2 / 2) times a
// polynomial in t = 1 / (1 + |z| / 5), fitted to the scaled tail erfcx / 2 with
// least largest relative error (1.3e-6 for |z| up to 14, where the tail has
// long left float16's range and is about to leave bfloat16's).  Evaluated in FP32
// it is 7e-6 off at |z| = 12 and 1.2e-5 at 13, from the rounding of z^2 / 2; the
// types round to 2^-9 and 2^-12.  One exponential and one quotient, where erff takes
// both of its branches in a warp.
__device__ __forceinline__ float normal_tail(float z, float &gauss) {
    const float a = fabsf(z);
    gauss = fast_exp2((-0.5f * kLog2E) * a * a);
    const float t = fast_reciprocal(fmaf(0.2f, a, 1.0f));
    float q = fmaf(t, 0.2790941894f, -0.3868259490f);
    q = fmaf(t, q, 0.4469392002f);
    q = fmaf(t, q, -0.1231861413f);
    q = fmaf(t, q, 0.1325369924f);
    q = fmaf(t, q, 0.0710921586f);
    q = fmaf(t, q, 0.0803501904f);
    return q * t * gauss;
}

// The same for FP32, with t = 1 / (1 + 0.4 |z|) (fit: 2e-8) and what rounding leaves of
// z^2 / 2 and of t put back: 6.5 x 2^-24 of the tail and expf's error, where (1 + erf) / 2
// cancels (at z = -5 it is 4 % off).  erfcf with the same correction is as exact and takes
// longer (1000 x 1030 x 777 with gelu, one call among others: 28.8 us for 25.7).  From
// |z| = 20 on the tail is 0; cut there, an infinity leaves no inf - inf.
__device__ __forceinline__ float normal_tail_f32(float z, float &gauss) {
    const float a = fminf(fabsf(z), 20.0f), h = 0.5f * a * a, e = expf(-h);
    gauss = fmaf(-e, fmaf(0.5f * a, a, -h), e);
    const float d = fmaf(0.4f, a, 1.0f);
    float t = fast_reciprocal(d);
    t = fmaf(t, fmaf(-d, t, 1.0f), t);
    // by pairs of powers: the chain is what an epilogue with few warps waits for
    const float t2 = t * t, t4 = t2 * t2;
    const float p0 = fmaf(t, 0.15963622927665710f, 0.15957549214363098f), p2 = fmaf(t, 0.09175224602222443f, 0.13305851817131042f);
    const float p4 = fmaf(t, 0.12209832668304443f, -0.02815046161413193f), p6 = fmaf(t, 0.38489249348640442f, -0.37734243273735046f);
    const float p8 = fmaf(t, 0.03242806717753410f, -0.17794845998287201f);
    const float q = fmaf(t4, fmaf(t4, p8, fmaf(t2, p6, p4)), fmaf(t2, p2, p0));
    return q * t * gauss;
}

// z Phi(z) from the tail; z - z tail would be a NaN at infinity.
__device__ __forceinline__ float gelu_of(float z, float tail) { return z * (z < 0.0f ? tail : 1.0f - tail); }
// A call of its own: the FP32 product's epilogue unrolls it 112 times beside as many
// accumulators, and inlined it took registers and instruction fetches from the rest
// (4096^3 573 us, as a call 510; with erff inlined 524, and 1000 x 1030 x 777 with the
// saved argument 37.3, 33 and 35.7).
static __device__ __noinline__ float gelu_f32(float z) {
    float gauss;
    return gelu_of(z, normal_tail_f32(z, gauss));
}

template <int ACT, bool EXACT>
__device__ __forceinline__ float activate(float z) {
    if constexpr (ACT == LINEAR_ACT_RELU) return z < 0.0f ? 0.0f : z;  // a NaN stays one
    if constexpr (ACT == LINEAR_ACT_SILU) return z * logistic<EXACT>(z);
    if constexpr (ACT == LINEAR_ACT_GELU) {
        if constexpr (EXACT) return gelu_f32(z);
        float gauss;
        return gelu_of(z, normal_tail(z, gauss));
    }
    if constexpr (ACT == LINEAR_ACT_GELU_TANH) return z * logistic<EXACT>(kGeluA * (z + kGeluB * z * z * z));
    return z;
}
// act'(z)
template <int ACT, bool EXACT>
__device__ __forceinline__ float slope(float z) {
    if constexpr (ACT == LINEAR_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if constexpr (ACT == LINEAR_ACT_SILU) {
        float pq;
        const float p = logistic<EXACT>(z, pq);
        return p + z * pq;
    }
    if constexpr (ACT == LINEAR_ACT_GELU) {
        float gauss;
        const float tail = EXACT ? normal_tail_f32(z, gauss) : normal_tail(z, gauss);
        return (z < 0.0f ? tail : 1.0f - tail) + z * kInvSqrt2Pi * gauss;
    }
    if constexpr (ACT == LINEAR_ACT_GELU_TANH) {
        float pq;
        const float p = logistic<EXACT>(kGeluA * (z + kGeluB * z * z * z), pq);
        const float c = fminf(fabsf(z), 100.0f);  // pq is 0 long before, and c * c stays finite
        return p + z * pq * kGeluA * (1.0f + 3.0f * kGeluB * c * c);
    }
    return 1.0f;
}

// f(tag) for the activation `act`, the tag's value a constant.
template <int V>
struct Int {
    static constexpr int value = V;
};
template <typename F>
__device__ __forceinline__ void with_activation(int act, F &&f) {
    switch (act) {
        case LINEAR_ACT_RELU: f(Int<LINEAR_ACT_RELU>{}); break;
        case LINEAR_ACT_SILU: f(Int<LINEAR_ACT_SILU>{}); break;
        case LINEAR_ACT_GELU: f(Int<LINEAR_ACT_GELU>{}); break;
        case LINEAR_ACT_GELU_TANH: f(Int<LINEAR_ACT_GELU_TANH>{}); break;
        default: f(Int<LINEAR_ACT_NONE>{}); break;
    }
}

}  // namespace lt
