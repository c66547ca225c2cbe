// gated_act.cuh -- the activations of the gated feed-forward block and their
// derivatives, in fp32.
//
// With s the logistic function, P the normal distribution and p its density:
//   silu       a = g s(g)                 a' = s (1 + g (1 - s))
//   gelu       a = g P(g)                 a' = P + g p(g)
//   gelu_tanh  a = g s(2z), z = sqrt(2/pi) (g + 0.044715 g^3): the form with tanh,
//              since 1 + tanh z = 2 s(2z), without its cancellation below zero
//              a' = s + 2 g s (1 - s) z'
//   relu       a = max(g, 0)              a' = 1 for g > 0, else 0
#pragma once

#include <cuda_runtime.h>

#include <type_traits>

#include "rra.h"

namespace rra {

// EXACT: for fp32 results.  16-bit ones are as near with the fast exponential and
// quotient: the exponential misses by 2 + 1.2 |g| units of its last place, the quotient
// by 2, together below 2^-16 of s as far as s is an fp32 number, and below 2^-18 where
// g s is one of fp16: a hundredth of the results' own half step.  Both sides of the
// quotient are quarters, exactly: it is 0 for denominators above 2^126, and those up to
// 2^128 (g down to -88.7) have results that bf16 holds.
template <bool EXACT> __device__ __forceinline__ float logistic(float g)
{
    if (EXACT)
        return 1.0f / (1.0f + expf(-g));
    return __fdividef(0.25f, fmaf(0.25f, __expf(-g), 0.25f));
}

constexpr float kGeluSlope = 1.5957691216057308f; // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

template <bool EXACT> __device__ __forceinline__ float gelu_logistic(float g)
{
    return logistic<EXACT>(kGeluSlope * fmaf(kGeluCubic * g * g, g, g));
}

// The activation is a template parameter where loops over many elements are
// unrolled: chosen for every element, its four codes are more than the instruction
// cache holds (gated_ff of 128 x 64 x 8192 bf16 took 19 us so, and takes 8).
template <int ACT, bool EXACT> __device__ __forceinline__ float act_value(float g)
{
    if constexpr (ACT == RRA_ACT_SILU)
        return g * logistic<EXACT>(g);
    else if constexpr (ACT == RRA_ACT_GELU)
        return g * normcdff(g);
    else if constexpr (ACT == RRA_ACT_GELU_TANH)
        return g * gelu_logistic<EXACT>(g);
    else
        return g > 0.0f || g != g ? g : 0.0f; // (NaN stays)
}

// a(g); *slope = a'(g).
template <int ACT, bool EXACT> __device__ __forceinline__ float act_both(float g, float *slope)
{
    if constexpr (ACT == RRA_ACT_SILU) {
        const float s = logistic<EXACT>(g);
        *slope = s * fmaf(g, 1.0f - s, 1.0f);
        return g * s;
    } else if constexpr (ACT == RRA_ACT_GELU) {
        const float p = normcdff(g), e = EXACT ? expf(-0.5f * g * g) : __expf(-0.5f * g * g);
        *slope = fmaf(g, 0.3989422804014327f * e, p);
        return g * p;
    } else if constexpr (ACT == RRA_ACT_GELU_TANH) {
        const float s = gelu_logistic<EXACT>(g);
        // g^3 of a finite g may be infinite where s (1 - s) is 0: the square is bounded, and
        // what is 0 is multiplied in ahead of z'
        const float dz = kGeluSlope * fmaf(3.0f * kGeluCubic, fminf(g * g, 1e30f), 1.0f);
        *slope = fmaf(g * (s * (1.0f - s)), dz, s);
        return g * s;
    } else {
        *slope = g > 0.0f ? 1.0f : 0.0f;
        return g > 0.0f || g != g ? g : 0.0f;
    }
}

// The code for one activation of the four, f(a constant of its number), in device code
// and on the host.
#define RRA_BY_ACT(act, f)                                                                       \
    switch (act) {                                                                               \
    case RRA_ACT_SILU:                                                                           \
        return f(std::integral_constant<int, RRA_ACT_SILU>());                                   \
    case RRA_ACT_GELU:                                                                           \
        return f(std::integral_constant<int, RRA_ACT_GELU>());                                   \
    case RRA_ACT_GELU_TANH:                                                                      \
        return f(std::integral_constant<int, RRA_ACT_GELU_TANH>());                              \
    default:                                                                                     \
        return f(std::integral_constant<int, RRA_ACT_RELU>());                                   \
    }
template <typename F> __device__ __forceinline__ auto by_act(int act, const F &f) { RRA_BY_ACT(act, f) }
template <typename F> auto host_by_act(int act, const F &f) { RRA_BY_ACT(act, f) }
#undef RRA_BY_ACT

template <bool EXACT> __device__ __forceinline__ float act_of(int act, float g)
{
    return by_act(act, [&](auto a) { return act_value<decltype(a)::value, EXACT>(g); });
}

} // namespace rra
