// Root-mean-square norm with the residual's addition, for gfx950:
//
//   h = x + res,  rstd = 1 / sqrt(mean_k h^2 + eps),  y = w h rstd
//   dh = rstd (w dy - xh mean_k(w dy xh)) + dres,  dw = sum over the rows of dy xh,  xh = h rstd
//
// Both directions read each input once and write each output once and are bound
// by that: a row stays in registers between its sum and its outputs (8 values
// per vector, up to 4 vectors per thread), rows of up to 2048 values in one wave,
// up to 8192 in 4 and up to 16384 in 16. The forward pass also gives y in 8 bits
// (codes and absmax of blocks of 64, the blockwise Int8 codec's) from the same
// registers, 8 neighbouring lanes holding a block. y and its 8-bit values come
// from h before its rounding to the residual's type: one rounding each.
// Sums are fp32 in a fixed order; dw is summed per workgroup over its rows, then
// over the workgroups.
#include "common.h"
#include "launch.h"

#include <type_traits>

namespace qlora {

namespace {

__device__ __forceinline__ void nm_load(const void* p, bool bf16, int64_t at, float* v) {
  if (bf16) {
    const u32x4_t w = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p) + at);
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(x[e] << 16);
      v[2 * e + 1] = __uint_as_float(x[e] & 0xFFFF0000u);
    }
  } else {
    const f32x4_t a = *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + at);
    const f32x4_t b = *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + at + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

__device__ __forceinline__ void nm_store(void* p, bool bf16, int64_t at, const float* v) {
  if (bf16) {
    *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p) + at) =
        u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
  } else {
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + at) = f32x4_t{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + at + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
  }
}

// The sum over the WAVES waves of a row; every thread of them gets it. red: one float per wave of the workgroup.
template <int WAVES>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if constexpr (WAVES > 1) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += red[w];
    __syncthreads();                               // red may be written again
  }
  return v;
}

// Workgroups of 4 waves (16 where a row takes 16): 4 rows at a time for WAVES = 1.
template <int WAVES>
struct NormShape {
  static constexpr int kThreads = WAVES == 16 ? 1024 : 256;
  static constexpr int kRows = kThreads / 64 / WAVES;
};

template <int WAVES, int NV>
__global__ __launch_bounds__(NormShape<WAVES>::kThreads) void norm_fwd_kernel(NormFwd c) {
  using S = NormShape<WAVES>;
  __shared__ float red[16];
  const int t = threadIdx.x % (64 * WAVES);
  const int64_t row = (int64_t)blockIdx.x * S::kRows + threadIdx.x / (64 * WAVES);
  if (WAVES == 1 && row >= c.M) return;            // whole waves; no barrier follows
  const int64_t base = row * c.K;
  float h[NV][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t k = (int64_t)(i * 64 * WAVES + t) * 8;
    if (k < c.K) {
      nm_load(c.x, c.x_bf16, base + k, h[i]);
      if (c.res) {
        float r[8];
        nm_load(c.res, c.res_bf16, base + k, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] += r[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(h[i][e], h[i][e], ss);
    }
  }
  const float rstd = 1.0f / __builtin_sqrtf(row_sum<WAVES>(ss, red) / (float)c.K + c.eps);
  if (c.rstd && t == 0) c.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t k = (int64_t)(i * 64 * WAVES + t) * 8;
    if (k >= c.K) continue;
    if (c.h) nm_store(c.h, c.res_bf16, base + k, h[i]);
    float y[8];
    if (c.w) {
      float w[8];
      nm_load(c.w, c.w_bf16, k, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = h[i][e] * rstd * w[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = h[i][e] * rstd;
    }
    if (c.y) nm_store(c.y, true, base + k, y);
    if (c.codes) {                                 // K % 64 == 0: the 8 lanes of a block agree
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = __builtin_fmaxf(m, __builtin_fabsf(y[e]));
      m = wave_max(m, 8);
      const float q = m < 0x1p-120f ? 0.0f : 127.0f / m;
      uint32_t b[2] = {0u, 0u};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = __builtin_fminf(__builtin_fmaxf(__builtin_rintf(y[e] * q), -127.0f), 127.0f);
        b[e >> 2] |= ((uint32_t)((int32_t)x) & 0xFFu) << (8 * (e & 3));
      }
      *reinterpret_cast<u32x2_t*>(c.codes + base + k) = u32x2_t{b[0], b[1]};
      if ((t & 7) == 0) c.absmax[(base + k) >> 6] = m;
    }
  }
}

// Rows first, first + rows in flight, ...: each group of WAVES waves sums dw over its rows into part[group].
template <int WAVES, int NV, bool DW>
__global__ __launch_bounds__(NormShape<WAVES>::kThreads) void norm_bwd_kernel(NormBwd c) {
  using S = NormShape<WAVES>;
  __shared__ float red[16];
  const int t = threadIdx.x % (64 * WAVES);
  const int64_t group = (int64_t)blockIdx.x * S::kRows + threadIdx.x / (64 * WAVES);
  const int64_t groups = (int64_t)gridDim.x * S::kRows;
  float dw[DW ? NV : 1][8];
  float w[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t k = (int64_t)(i * 64 * WAVES + t) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[i][e] = 1.0f;
      if constexpr (DW) dw[i][e] = 0.0f;
    }
    if (c.w && k < c.K) nm_load(c.w, c.w_bf16, k, w[i]);
  }
  for (int64_t row = group; row < c.M; row += groups) {   // uniform for the waves of a row
    const int64_t base = row * c.K;
    const float rstd = c.rstd[row];
    float xh[NV][8], dy[NV][8], dr[NV][8];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t k = (int64_t)(i * 64 * WAVES + t) * 8;
      if (k >= c.K) continue;
      nm_load(c.h, c.h_bf16, base + k, xh[i]);
      nm_load(c.dy, true, base + k, dy[i]);
      if (c.dres) nm_load(c.dres, c.h_bf16, base + k, dr[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xh[i][e] *= rstd;
        if constexpr (DW) dw[i][e] = __builtin_fmaf(dy[i][e], xh[i][e], dw[i][e]);
        dy[i][e] *= w[i][e];
        sum = __builtin_fmaf(dy[i][e], xh[i][e], sum);
      }
    }
    const float mean = row_sum<WAVES>(sum, red) / (float)c.K;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t k = (int64_t)(i * 64 * WAVES + t) * 8;
      if (k >= c.K) continue;
      float d[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[e] = rstd * (dy[i][e] - xh[i][e] * mean);
        if (c.dres) d[e] += dr[i][e];
      }
      nm_store(c.dh, c.h_bf16, base + k, d);
      if (c.dx16) nm_store(c.dx16, true, base + k, d);
    }
  }
  if constexpr (DW) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t k = (int64_t)(i * 64 * WAVES + t) * 8;
      if (k < c.K) nm_store(c.part, false, group * c.K + k, dw[i]);
    }
  }
}

// dw[k] = the groups' sums, 16 parts of the groups in order, then the parts in order. 64 columns per workgroup.
__global__ __launch_bounds__(1024) void norm_dw_kernel(const float* __restrict__ part, int groups, int64_t K, float* __restrict__ dw) {
  __shared__ float red[16][64];
  const int c = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int64_t k = (int64_t)blockIdx.x * 64 + c;
  const int per = (groups + 15) / 16, lo = q * per, hi = lo + per < groups ? lo + per : groups;
  float v = 0.0f;
  if (k < K)
    for (int g = lo; g < hi; ++g) v += part[(int64_t)g * K + k];
  red[q][c] = v;
  __syncthreads();
  if (q == 0 && k < K) {
#pragma unroll
    for (int i = 1; i < 16; ++i) v += red[i][c];
    dw[k] = v;
  }
}

template <typename F>
hipError_t by_shape(int64_t K, F&& go) {
  const int64_t n8 = (K + 7) / 8;
  auto nv = [&](auto waves, int64_t per) -> hipError_t {
    const int64_t n = (n8 + per - 1) / per;
    if constexpr (decltype(waves)::value == 16) {
      return go(waves, std::integral_constant<int, 2>{});   // above 8192: two vectors
    } else {
      if (n <= 1) return go(waves, std::integral_constant<int, 1>{});
      if (n == 2) return go(waves, std::integral_constant<int, 2>{});
      if (n == 3) return go(waves, std::integral_constant<int, 3>{});
      return go(waves, std::integral_constant<int, 4>{});
    }
  };
  if (n8 <= 4 * 64) return nv(std::integral_constant<int, 1>{}, 64);
  if (n8 <= 4 * 256) return nv(std::integral_constant<int, 4>{}, 256);
  return nv(std::integral_constant<int, 16>{}, 1024);
}

}  // namespace

hipError_t launch_norm_fwd(const NormFwd& c, hipStream_t stream) {
  if (c.M == 0) return hipSuccess;
  return by_shape(c.K, [&](auto waves, auto nv) {
    using S = NormShape<decltype(waves)::value>;
    hipLaunchKernelGGL((norm_fwd_kernel<decltype(waves)::value, decltype(nv)::value>),
                       dim3((unsigned)((c.M + S::kRows - 1) / S::kRows)), dim3(S::kThreads), 0, stream, c);
    return hipGetLastError();
  });
}

// Groups of waves that sum dw: four workgroups per CU.
int norm_slices(int64_t M) {
  const int64_t most = 4 * (int64_t)device_cu_count();
  return (int)((M < most ? M : most) + 3) / 4 * 4;
}

hipError_t launch_norm_bwd(const NormBwd& c, hipStream_t stream) {
  const int groups = norm_slices(c.M);
  hipError_t e = hipSuccess;
  if (c.M > 0) e = by_shape(c.K, [&](auto waves, auto nv) {
    using S = NormShape<decltype(waves)::value>;
    const dim3 grid((unsigned)((groups + S::kRows - 1) / S::kRows));
    if (c.dw)
      hipLaunchKernelGGL((norm_bwd_kernel<decltype(waves)::value, decltype(nv)::value, true>), grid, dim3(S::kThreads), 0, stream, c);
    else
      hipLaunchKernelGGL((norm_bwd_kernel<decltype(waves)::value, decltype(nv)::value, false>), grid, dim3(S::kThreads), 0, stream, c);
    return hipGetLastError();
  });
  if (e != hipSuccess || !c.dw) return e;
  hipLaunchKernelGGL(norm_dw_kernel, dim3((unsigned)((c.K + 63) / 64)), dim3(1024), 0, stream, c.part, groups, c.K, c.dw);
  return hipGetLastError();
}

}  // namespace qlora
