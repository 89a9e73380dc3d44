// The activations of the gated feed-forward block and their derivatives, in fp32.
//   silu: f = g p, p = 1 / (1 + exp(-g));                     f' = p + f (1 - p)
//   gelu (tanh form): 0.5 g (1 + tanh(z / 2)) = g p, p = 1 / (1 + exp(-z)),
//         z = 2 sqrt(2/pi) (g + 0.044715 g^3);                f' = p + f (1 - p) z'
// The exponential and the reciprocal are the hardware's (about one fp32 ulp each, the exponent's
// product with log2 e adds |z| 2^-24): errors near 2^-20, against the output's 2^-11. exp
// overflowing to infinity gives p = 0.
#pragma once

#include "device_common.h"

namespace awq {

enum GatedAct { kSilu = 0, kGelu = 1 };

template <int ACT>
__device__ __forceinline__ float act_p(float g) {
  constexpr float kLog2e = 1.4426950408889634f;
  constexpr float kC = 1.5957691216057308f;   // 2 sqrt(2 / pi)
  const float z = ACT == kSilu ? g : kC * __builtin_fmaf(0.044715f * g * g, g, g);
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * z));
}

template <int ACT>
__device__ __forceinline__ float act_f(float g) {
  return g * act_p<ACT>(g);
}

// f and f'
template <int ACT>
__device__ __forceinline__ float act_f_df(float g, float& df) {
  constexpr float kC = 1.5957691216057308f;
  const float p = act_p<ACT>(g), f = g * p;
  const float q = f * (1.0f - p);
  df = ACT == kSilu ? p + q : __builtin_fmaf(q, kC * __builtin_fmaf(0.134145f * g, g, 1.0f), p);
  return f;
}

}  // namespace awq
