// gated_act.cuh -- the activations of the gated feed-forward block and their
// derivatives, in fp32.
//
// With s the logistic function, P the normal distribution and p its density:
//   silu       a = g s(g)                 a' = s (1 + g (1 - s))
//   gelu       a = g P(g)                 a' = P + g p(g)
//   gelu_tanh  a = g s(2z), z = sqrt(2/pi) (g + 0.044715 g^3): the form with tanh,
//              since 1 + tanh z = 2 s(2z), without its cancellation below zero
//              a' = s (1 + 2 g (1 - s) z')
//   relu       a = max(g, 0)              a' = 1 for g > 0, else 0
#pragma once

#include <cuda_runtime.h>

#include "rra.h"

namespace rra {

// EXACT: for fp32 results.  16-bit ones are as near with the fast exponential and
// quotient, whose errors (2^-21) are a 1000th of a half step of theirs.
template <bool EXACT> __device__ __forceinline__ float logistic(float g)
{
    if (EXACT)
        return 1.0f / (1.0f + expf(-g));
    return __fdividef(1.0f, 1.0f + __expf(-g));
}

constexpr float kGeluSlope = 1.5957691216057308f; // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

template <bool EXACT> __device__ __forceinline__ float gelu_logistic(float g)
{
    return logistic<EXACT>(kGeluSlope * fmaf(kGeluCubic * g * g, g, g));
}

template <bool EXACT> __device__ __forceinline__ float act_value(int act, float g)
{
    switch (act) {
    case RRA_ACT_SILU:
        return g * logistic<EXACT>(g);
    case RRA_ACT_GELU:
        return g * normcdff(g);
    case RRA_ACT_GELU_TANH:
        return g * gelu_logistic<EXACT>(g);
    default:
        return g > 0.0f || g != g ? g : 0.0f; // (NaN stays)
    }
}

// a(g); *slope = a'(g).
template <bool EXACT> __device__ __forceinline__ float act_both(int act, float g, float *slope)
{
    switch (act) {
    case RRA_ACT_SILU: {
        const float s = logistic<EXACT>(g);
        *slope = s * fmaf(g, 1.0f - s, 1.0f);
        return g * s;
    }
    case RRA_ACT_GELU: {
        const float p = normcdff(g), e = EXACT ? expf(-0.5f * g * g) : __expf(-0.5f * g * g);
        *slope = fmaf(g, 0.3989422804014327f * e, p);
        return g * p;
    }
    case RRA_ACT_GELU_TANH: {
        const float s = gelu_logistic<EXACT>(g);
        // (the square of a finite g may be infinite where 1 - s is 0)
        const float dz = kGeluSlope * fmaf(3.0f * kGeluCubic, fminf(g * g, 1e30f), 1.0f);
        *slope = s * fmaf(g * (1.0f - s), dz, 1.0f);
        return g * s;
    }
    default:
        *slope = g > 0.0f ? 1.0f : 0.0f;
        return g > 0.0f || g != g ? g : 0.0f;
    }
}

} // namespace rra
