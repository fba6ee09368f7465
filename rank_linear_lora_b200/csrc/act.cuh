// act.cuh -- the activations of the gated and the epilogue projections, and their
// derivatives, in fp32.
//
//   relu       max(v, 0)                              derivative 1 for v > 0, else 0
//   silu       v s(v), s(v) = 1 / (1 + e^-v)          s (1 + v (1 - s))
//   gelu       v P(v), P the normal distribution      P(v) + v p(v), p its density
//   gelu_tanh  v/2 (1 + tanh z) = v s(2z),            s(2z) (1 + v (1 - s(2z)) 2 z'),
//              z = c (v + 0.044715 v^3), c = sqrt(2/pi)   z' = c (1 + 3 * 0.044715 v^2)
//
// gelu's P(v) = 1 - P(-v) comes from erfc(z) = e^-z^2 t(a1 + t(a2 + ... + t a6)), t = 1 / (1 + p z),
// z >= 0: the polynomial is this file's own fit of e^z^2 erfc(z) over 0 <= z <= 9.3 (where e^-z^2
// leaves fp32), the one of smallest relative error: 4e-6.  It shares its exponential with the
// density and costs about half of erff.  The relative error matters on the negative side, where P
// is as small as its tail: v P(v) is off by less than 2^-15 of itself down to v = -12.5, far inside
// one bf16 rounding (a fit of smallest absolute error, 1.5e-7, has every digit wrong there).
// The logistic function goes through __expf and __fdividef (a few units in the last place of
// fp32, far inside the one bf16 rounding that every result takes); at the ends, e^-v above 2^126
// (v < -87.3) gives s = 0, for which silu is 0 and not v e^v, 1e-36 and less, and e^-v = 0 gives
// s = 1.  NaN stays NaN in each of them.
#pragma once

#include <cuda_runtime.h>

#include "../../include/lora_linear.h"

namespace lora {

template <int A>
struct ActCode {
    static constexpr int value = A;
};

// f(ActCode<act>()) for the run-time code `act` (validated on the host).
template <class F>
__device__ __forceinline__ void act_dispatch(int act, F &&f) {
    switch (act) {
        case LORA_ACT_RELU: f(ActCode<LORA_ACT_RELU>()); break;
        case LORA_ACT_SILU: f(ActCode<LORA_ACT_SILU>()); break;
        case LORA_ACT_GELU: f(ActCode<LORA_ACT_GELU>()); break;
        case LORA_ACT_GELU_TANH: f(ActCode<LORA_ACT_GELU_TANH>()); break;
        default: f(ActCode<LORA_ACT_NONE>()); break;
    }
}

__device__ __forceinline__ float logistic(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

constexpr float GELU_C2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float GELU_A = 0.044715f;
constexpr float INV_SQRT2 = 0.70710678118654752f, INV_SQRT_2PI = 0.39894228040143268f;

// P(v) of the normal distribution; `e` = e^(-v^2 / 2).
__device__ __forceinline__ float normal_cdf(float v, float &e) {
    const float z = fabsf(v) * INV_SQRT2;
    e = __expf(-z * z);
    const float t = __fdividef(1.0f, 1.0f + 0.4344f * z);
    const float tail = 0.276168525f + t * (0.00657896465f + t * (0.387573302f + t * -0.152294233f));
    const float half_erfc = 0.5f * e * t * (0.245644301f + t * (0.236326128f + t * tail));
    return v < 0.0f ? half_erfc : 1.0f - half_erfc;
}

template <int A>
__device__ __forceinline__ float act_value(float v) {
    if constexpr (A == LORA_ACT_RELU) return v < 0.0f ? 0.0f : v;  // NaN stays
    if constexpr (A == LORA_ACT_SILU) return __fdividef(v, 1.0f + __expf(-v));
    if constexpr (A == LORA_ACT_GELU) {
        float e;
        return v * normal_cdf(v, e);
    }
    if constexpr (A == LORA_ACT_GELU_TANH)
        return __fdividef(v, 1.0f + __expf(-GELU_C2 * (v + GELU_A * v * v * v)));
    return v;
}

// act(v) and act'(v).
template <int A>
__device__ __forceinline__ void act_both(float v, float &y, float &dy) {
    if constexpr (A == LORA_ACT_RELU) {
        y = v < 0.0f ? 0.0f : v;
        dy = v > 0.0f ? 1.0f : 0.0f;
    } else if constexpr (A == LORA_ACT_SILU) {
        const float s = logistic(v);
        y = v * s;
        dy = s * (1.0f + v * (1.0f - s));
    } else if constexpr (A == LORA_ACT_GELU) {
        float e;
        const float cdf = normal_cdf(v, e);
        y = v * cdf;
        dy = cdf + v * INV_SQRT_2PI * e;
    } else if constexpr (A == LORA_ACT_GELU_TANH) {
        // beyond |v| = 100 s is exactly 0 or 1 and the derivative with it; the bound keeps
        // 0 * v^3 from becoming 0 * inf
        const float b = fabsf(v) > 100.0f ? copysignf(100.0f, v) : v;
        const float s = logistic(GELU_C2 * (b + GELU_A * b * b * b));
        y = v * s;
        dy = s * (1.0f + b * (1.0f - s) * GELU_C2 * (1.0f + 3.0f * GELU_A * b * b));
    } else {
        y = v;
        dy = 1.0f;
    }
}

}  // namespace lora
