// dq4_linear_device.h -- device pieces shared by the fused linear and gated
// feed-forward sources (internal; not part of the C ABI): the 16-bit types,
// the activations and the operand layout of the matrix instruction.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "dq4_device.h"
#include "dq4_linear.h"

#pragma clang fp contract(off)

namespace dq4 {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// The 16-bit type T of a call (OUT = DQ4_F16 or DQ4_BF16): conversions from
// FP32 are one round-to-nearest-even step of a rounded FP32 value, and the
// products run on v_mfma_f32_16x16x32_{f16,bf16}: D (16 x 16, FP32) += A (16
// x 32) B (32 x 16).  Lane l holds A[l % 16][8 (l / 16) .. + 7] and
// B[8 (l / 16) .. + 7][l % 16], and D[4 (l / 16) + i][l % 16] for i = 0 .. 3.
template <int OUT>
struct Half;

template <>
struct Half<DQ4_F16> {
    typedef f16x8 Frag;
    static __device__ __forceinline__ float widen(uint32_t bits16)
    {
        return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits16)));
    }
    static __device__ __forceinline__ uint32_t pack2(float lo, float hi)
    {
        // one v_cvt_pk_f16_f32, round to nearest even
        return __builtin_bit_cast(
            uint32_t, __builtin_convertvector((f32x2{rounded_fp32(lo), rounded_fp32(hi)}), f16x2));
    }
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(Frag, a),
                                                      __builtin_bit_cast(Frag, b), c, 0, 0, 0);
    }
};

template <>
struct Half<DQ4_BF16> {
    typedef bf16x8 Frag;
    static __device__ __forceinline__ float widen(uint32_t bits16)
    {
        return __builtin_bit_cast(float, bits16 << 16);
    }
    static __device__ __forceinline__ uint32_t pack2(float lo, float hi)
    {
        // one v_cvt_pk_bf16_f32, round to nearest even
        return __builtin_bit_cast(
            uint32_t, __builtin_convertvector((f32x2{rounded_fp32(lo), rounded_fp32(hi)}), bf16x2));
    }
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(Frag, a),
                                                       __builtin_bit_cast(Frag, b), c, 0, 0, 0);
    }
};

// ---------------------------------------------------------------------------
// activations, in FP32
// ---------------------------------------------------------------------------
// exp(x) as 2^(x log2 e): the rounding of x log2 e leaves a relative error of
// about |x| 2^-24, at most 6e-6 where the result is a normal FP32 number, far
// below the half step of FP16 or BF16 that the results are rounded to (the
// bias gradient, in FP32, keeps it).
__device__ __forceinline__ float exp_f32(float x)
{
    return __builtin_amdgcn_exp2f(x * 1.44269504088896341f);
}

// 1 / (1 + exp(-x)); the reciprocal instruction is within 1 ulp.
__device__ __forceinline__ float sigmoid_f32(float x)
{
    return __builtin_amdgcn_rcpf(1.0f + exp_f32(-x));
}

// erfc(|x|): the Chebyshev fit t exp(-x^2 + P(t)), t = 1 / (1 + |x| / 2), of
// Press, Teukolsky, Vetterling and Flannery, "Numerical Recipes" (erfcc).  The
// fit's own relative error is below 1.2e-7; here the exponent, about x^2 in
// size, is rounded three times, which adds up to 1.5 x^2 2^-23 (1.5e-5 at x =
// 9), and results below 2^-126, from |x| = 9.2 on, are flushed to 0.
__device__ __forceinline__ float erfc_abs_f32(float x)
{
    const float z = __builtin_fabsf(x);
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.5f * z);
    float p = 0.17087277f;
    p = -0.82215223f + t * p;
    p = 1.48851587f + t * p;
    p = -1.13520398f + t * p;
    p = 0.27886807f + t * p;
    p = -0.18628806f + t * p;
    p = 0.09678418f + t * p;
    p = 0.37409196f + t * p;
    p = 1.00002368f + t * p;
    p = -1.26551223f + t * p;
    return t * exp_f32(-z * z + p);
}

// The normal distribution's integral, erfc(-z / sqrt 2) / 2.
__device__ __forceinline__ float normal_cdf_f32(float z)
{
    const float half_tail = 0.5f * erfc_abs_f32(z * 0.70710678118654752f);
    return z > 0.0f ? 1.0f - half_tail : half_tail;
}

constexpr float kGeluTwoC = 1.59576912160573071f;     // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

// The tanh form's 2 v, v = sqrt(2/pi) (z + 0.044715 z^3), with z held to [-64,
// 64]: the sigmoid is 0 or 1 long before that, and z^3 cannot overflow.  A NaN
// gives -64: what is computed from it has to take the NaN from z itself.
__device__ __forceinline__ float gelu_clamp(float z)
{
    return __builtin_amdgcn_fmed3f(z, -64.0f, 64.0f);
}

// z held to [-bound, bound]; a NaN stays.
__device__ __forceinline__ float held(float z, float bound)
{
    return z != z ? z : __builtin_amdgcn_fmed3f(z, -bound, bound);
}

// act(z); z/2 (1 + tanh v) is z sigmoid(2 v).
__device__ __forceinline__ float act_f32(int act, float z)
{
    switch (act) {
    case DQ4_ACT_RELU:
        return z < 0.0f ? 0.0f : z;
    case DQ4_ACT_SILU:
        return z * sigmoid_f32(z);
    case DQ4_ACT_GELU:
        return z * normal_cdf_f32(z);
    case DQ4_ACT_GELU_TANH: {
        const float c = gelu_clamp(z);
        return z * sigmoid_f32(kGeluTwoC * (c + kGeluCubic * (c * c * c)));
    }
    default:
        return z;
    }
}

// act(z) and its derivative, for a saved z: a NaN gives NaN, and the
// infinities, which a 16-bit z reaches by overflow, give the limits (the
// formulas alone give 0 times infinity there).  `c` is z with the infinities
// held to the largest finite number, whose products with a vanished sigmoid or
// density are 0; z itself is multiplied only where it is not negative infinity.
__device__ __forceinline__ void act_and_slope_f32(int act, float z, float *value, float *slope)
{
    constexpr float kMax = 3.402823466e+38f;
    switch (act) {
    case DQ4_ACT_RELU:
        *value = z < 0.0f ? 0.0f : z;
        *slope = z > 0.0f ? 1.0f : z != z ? z : 0.0f;
        return;
    case DQ4_ACT_SILU: {
        const float s = sigmoid_f32(z), c = held(z, kMax);
        *value = (z > 0.0f ? z : c) * s;
        *slope = s * (1.0f + c * (1.0f - s));
        return;
    }
    case DQ4_ACT_GELU: {
        const float p = normal_cdf_f32(z), c = held(z, kMax);
        *value = (z > 0.0f ? z : c) * p;
        *slope = p + c * (kInvSqrt2Pi * exp_f32(-0.5f * (z * z)));
        return;
    }
    case DQ4_ACT_GELU_TANH: {
        const float c = held(z, 64.0f);
        const float s = sigmoid_f32(kGeluTwoC * (c + kGeluCubic * (c * c * c)));
        *value = (z > 0.0f ? z : c) * s;
        *slope = s + c * s * (1.0f - s) * (kGeluTwoC * (1.0f + 3.0f * kGeluCubic * (c * c)));
        return;
    }
    default:
        *value = z;
        *slope = 1.0f;
        return;
    }
}

}  // namespace dq4
