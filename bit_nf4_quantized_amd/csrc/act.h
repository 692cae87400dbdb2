// The gated block's activations, act(g) = g sigma(z): z = g (SiLU) or
// z = sqrt(8 / pi) (g + 0.044715 g^3) (GELU in its tanh form), in fp32.
#pragma once

#include "common.h"
#include "launch.h"

namespace qlora {

template <int ACT>
__device__ __forceinline__ float act_of(float g) {
  const float z = ACT == kActSilu ? g : 1.5957691216057308f * (g + 0.044715f * (g * g * g));
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

// act(g) and act'(g) = sigma + g sigma (1 - sigma) dz/dg; sigma (1 - sigma) is 0
// for large |z|, where dz/dg may be infinite.
template <int ACT>
__device__ __forceinline__ void act_both(float g, float* a, float* d) {
  const float z = ACT == kActSilu ? g : 1.5957691216057308f * (g + 0.044715f * (g * g * g));
  const float p = __builtin_amdgcn_rcpf(1.0f + __expf(-z));
  const float q = p * (1.0f - p);
  const float dz = ACT == kActSilu ? 1.0f : 1.5957691216057308f * (1.0f + 0.134145f * (g * g));
  *a = g * p;
  *d = q == 0.0f ? p : p + g * q * dz;
}

}  // namespace qlora
