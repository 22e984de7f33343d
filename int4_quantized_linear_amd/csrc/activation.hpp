// activation.hpp -- the activations of the fused linears and their derivatives, in fp32 (gfx950).
// Codes are the CONVROT_ACT_* values of include/convrot.h.  The code is uniform over a launch, so
// each switch is a scalar branch.
//
// silu(z) = z s(z) and the tanh form of gelu, z (1 + tanh v) / 2 = z s(2v), share the logistic
// s(t) = 1 / (1 + e^-t), taken as one v_exp_f32 and one v_rcp_f32 (1 ulp each; e^-t rounds its
// argument once, so the relative error is about |t| 2^-24 + 3 ulp, far below the bf16 the result is
// rounded to).  At t -> -inf, e^-t is infinite and s is 0; at t -> +inf s is 1.
// At z = -inf (a channel masked through its bias; the lowest fp32 numbers round to it in a bf16 pre) and
// z = +inf every value and slope is its limit: a factor that would be infinite beside a zero is held
// at the largest finite number.  Each such min or max stands beside a term that is NaN for a NaN z, so NaN
// is kept.
// gelu(z) = max(z, 0) - |z| h(|z|) with h(a) = erfc(a / sqrt 2) / 2 the normal distribution's tail, so
// its negative side keeps its relative precision.  h(a) = e^(-a^2 / 2) t Q(t) with t = 1 / (1 + 0.28 a):
// erfcx(a / sqrt 2) / 2 falls like 1 / a, and Q, a polynomial of degree 8 fitted here for the least
// largest relative error over a in [0, 1e8] (1.5e-7; 4.4e-7 when evaluated in fp32), takes up the
// rest.  The device library's erfcf costs three times as much: the 4096 x 5376 x 16128 linear took
// 349 us with it, against 286 us with the tanh form.
#pragma once
#include <hip/hip_runtime.h>

namespace convrot {

constexpr int kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4;

constexpr float kMax = 3.40282347e38f;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhA = 1.59576912160573071f;               // 2 sqrt(2 / pi)
constexpr float kTanhB = 0.044715f * 1.59576912160573071f;

__device__ __forceinline__ float logistic(float t)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * t));
}

// s(t), and s(-t) = e^-t s(t) with the same exponential, so the two keep their relative precision on both
// sides.  Where e^-t overflows s(t) is 0 and rest 0 too, not 1: it is only ever multiplied by s(t).
__device__ __forceinline__ float logistic(float t, float &rest)
{
    const float e = __builtin_amdgcn_exp2f(-kLog2e * t), p = __builtin_amdgcn_rcpf(1.0f + e);
    rest = __builtin_fminf(e, kMax) * p;
    return p;
}

// h(|z|), and e^(-z^2 / 2) for the density.
__device__ __forceinline__ float normal_tail(float z, float &e)
{
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.28f, __builtin_fabsf(z), 1.0f));
    e = __builtin_amdgcn_exp2f((-0.5f * kLog2e * z) * z);
    float q = 0.0247895472f;
    q = __builtin_fmaf(q, t, -0.0938178039f);
    q = __builtin_fmaf(q, t, 0.0926928233f);
    q = __builtin_fmaf(q, t, -0.00657380259f);
    q = __builtin_fmaf(q, t, 0.0727781769f);
    q = __builtin_fmaf(q, t, 0.0836467225f);
    q = __builtin_fmaf(q, t, 0.103080311f);
    q = __builtin_fmaf(q, t, 0.111700095f);
    q = __builtin_fmaf(q, t, 0.111703855f);
    return q * t * e;
}

__device__ __forceinline__ float act_value(float z, int act)
{
    switch (act) {
    case kActRelu: return z < 0.0f ? 0.0f : z;                // keeps a NaN
    case kActSilu: return __builtin_fmaxf(z, -kMax) * logistic(z);
    case kActGelu: {
        float e;
        return __builtin_fmaf(-__builtin_fminf(__builtin_fabsf(z), kMax), normal_tail(z, e), z < 0.0f ? 0.0f : z);
    }
    case kActGeluTanh: return __builtin_fmaxf(z, -kMax) * logistic(z * __builtin_fmaf(kTanhB * z, z, kTanhA));
    default: return z;
    }
}

// act of 8 values in place: one branch for all of them, so that their exponential and reciprocal
// chains overlap (a branch per value serialises them).
__device__ __forceinline__ void act_values(float (&v)[8], int act)
{
#define CONVROT_ACT_CASE(code)                                                        \
    case code:                                                                        \
        _Pragma("unroll") for (int i = 0; i < 8; ++i) v[i] = act_value(v[i], code);   \
        break;
    switch (act) {
        CONVROT_ACT_CASE(kActRelu)
        CONVROT_ACT_CASE(kActSilu)
        CONVROT_ACT_CASE(kActGelu)
        CONVROT_ACT_CASE(kActGeluTanh)
    default: break;
    }
#undef CONVROT_ACT_CASE
}

// act(z) and act'(z) together.
//   silu': p + z p (1 - p);  gelu': Phi(z) + z phi(z);  gelu_tanh': p + z p (1 - p) (2v)'
// with 1 - p = s(-t), so nothing cancels.  (2v)' grows as z^2 while p (1 - p) is 0 in fp32 beyond
// |z| = 10, and z phi(z) beyond 15, so both hold z there before it could give inf * 0.  One exponential
// and one reciprocal serve both (2048 tokens' gated block backward 1420 -> 1398 us against two of each).
__device__ __forceinline__ void act_value_slope(float z, int act, float &value, float &slope)
{
    switch (act) {
    case kActRelu:
        value = z < 0.0f ? 0.0f : z;
        slope = z > 0.0f ? 1.0f : 0.0f;
        break;
    case kActSilu: {
        float rest;
        const float p = logistic(z, rest);
        value = __builtin_fmaxf(z, -kMax) * p;
        slope = __builtin_fmaf(__builtin_fminf(value, kMax), rest, p);
        break;
    }
    case kActGelu: {
        float e;
        const float h = normal_tail(z, e);
        value = __builtin_fmaf(-__builtin_fminf(__builtin_fabsf(z), kMax), h, z < 0.0f ? 0.0f : z);
        const float c = __builtin_fminf(__builtin_fmaxf(z, -16.0f), 16.0f);
        slope = __builtin_fmaf(c * kInvSqrt2Pi, e, z < 0.0f ? h : 1.0f - h);
        break;
    }
    case kActGeluTanh: {
        float rest;
        const float p = logistic(z * __builtin_fmaf(kTanhB * z, z, kTanhA), rest);
        value = __builtin_fmaxf(z, -kMax) * p;
        const float c = __builtin_fminf(__builtin_fmaxf(z, -16.0f), 16.0f);
        slope = __builtin_fmaf(c * p * rest, __builtin_fmaf(3.0f * kTanhB * c, c, kTanhA), p);
        break;
    }
    default:
        value = z;
        slope = 1.0f;
    }
}

// The same of N values: v becomes act(v), slope act'(v).
template <int N>
__device__ __forceinline__ void act_values_slopes(float (&v)[N], float (&slope)[N], int act)
{
#define CONVROT_ACT_CASE(label, code)                                                             \
    label:                                                                                        \
        _Pragma("unroll") for (int i = 0; i < N; ++i) act_value_slope(v[i], code, v[i], slope[i]); \
        break;
    switch (act) {
        CONVROT_ACT_CASE(case kActRelu, kActRelu)
        CONVROT_ACT_CASE(case kActSilu, kActSilu)
        CONVROT_ACT_CASE(case kActGelu, kActGelu)
        CONVROT_ACT_CASE(case kActGeluTanh, kActGeluTanh)
        CONVROT_ACT_CASE(default, kActNone)
    }
#undef CONVROT_ACT_CASE
}

} // namespace convrot
