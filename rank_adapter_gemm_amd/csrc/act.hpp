// The activations.
#pragma once

#include "common.hpp"

namespace lora {

// The logistic function of x; FINE uses the exact exponential and division
// (fp32 outputs), else one v_exp and one v_rcp (1 ulp each, far below bf16's
// step).  exp overflows to infinity for very negative x, which gives 0.
template <bool FINE> __device__ __forceinline__ float logistic(float x) {
    if (FINE) return 1.0f / (1.0f + expf(-x));
    return __builtin_amdgcn_rcpf(1.0f + __expf(-x));
}

constexpr float kGeluTanhK = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluTanhC = 0.044715f;

// silu: x q, q = logistic(x).  gelu: x cdf(x), the normal distribution's cdf
// by erfc, which keeps the small values of negative x.  gelu_tanh: 0.5 x (1 +
// tanh(z)) = x logistic(2 z), z = sqrt(2/pi) (x + 0.044715 x^3).
template <bool FINE> __device__ __forceinline__ float act_value(int act, float x) {
    if (act == LORA_ACT_SILU) return x * logistic<FINE>(x);
    if (act == LORA_ACT_GELU) return x * (0.5f * erfcf(-0.70710678118654752f * x));
    return x * logistic<FINE>(kGeluTanhK * fmaf(kGeluTanhC * x * x, x, x));
}

// The same with LORA_ACT_NONE.
template <bool FINE> __device__ __forceinline__ float act_or_none(int act, float x) {
    return act == LORA_ACT_NONE ? x : act_value<FINE>(act, x);
}

}  // namespace lora
