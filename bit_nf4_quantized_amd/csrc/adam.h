// Arithmetic shared by the optimiser kernels: the Adam update of one element,
// the fixed-order sums behind the gradient norm, and the clip coefficient.
#pragma once

#include <math.h>

#include "common.h"
#include "launch.h"

namespace qlora {

constexpr int kNormBlocks = 1024;

__device__ __forceinline__ double tree_sum_256(double v, double* s) {
  const int t = threadIdx.x;
  s[t] = v;
  __syncthreads();
  for (int w = 128; w > 0; w >>= 1) {
    if (t < w) s[t] += s[t + w];
    __syncthreads();
  }
  return s[0];
}

struct AdamConsts {
  float lr, b1, b2, omb1, omb2, eps, wd, bc1, bc2;
};

inline AdamConsts adam_consts(const AdamHyper& h) {
  AdamConsts k;
  k.lr = h.lr; k.b1 = h.beta1; k.b2 = h.beta2; k.eps = h.eps; k.wd = h.wd;
  k.omb1 = (float)(1.0 - (double)h.beta1);
  k.omb2 = (float)(1.0 - (double)h.beta2);
  k.bc1 = (float)(1.0 - pow((double)h.beta1, (double)h.step));
  k.bc2 = (float)(1.0 - pow((double)h.beta2, (double)h.step));
  return k;
}

__device__ __forceinline__ void adam_one(float& th, float g, float& m, float& v, float cf, const AdamConsts& k) {
  const float gc = cf * g;
  m = k.b1 * m + k.omb1 * gc;
  v = k.b2 * v + k.omb2 * (gc * gc);
  const float mh = m / k.bc1;
  const float vh = v / k.bc2;
  const float upd = mh / (__builtin_sqrtf(vh) + k.eps);
  th = th - k.lr * (upd + k.wd * th);
}

// norm and clip coefficient from the kNormBlocks partial sums of squares
static __global__ __launch_bounds__(1024) void clip_finalize_kernel(const double* __restrict__ part, double max_norm,
                                                             float* __restrict__ coef, double* __restrict__ norm) {
  __shared__ double s[1024];
  const int t = threadIdx.x;
  s[t] = part[t];
  __syncthreads();
  for (int w = 512; w > 0; w >>= 1) {
    if (t < w) s[t] += s[t + w];
    __syncthreads();
  }
  if (t == 0) {
    const double nrm = sqrt(s[0]);
    const double c = max_norm / (nrm + 1e-6);
    if (coef) *coef = (float)(c < 1.0 ? c : 1.0);
    if (norm) *norm = nrm;
  }
}

}  // namespace qlora
