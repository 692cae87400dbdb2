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
// over the workgroups. 8192 x 4096, bf16 onto an fp32 stream, with both outputs:
// 86 us, 5.1 TB/s (a large copy: 5.05). Backward, 8192 x 4096 on an fp32 stream: 88 us
// (5.4 TB/s) and 7.4 for dw's sum; 1001 x 6656 in bf16: 14.7 us (3.6 TB/s, the latency
// of one or two rows per workgroup) and 4.4.
#include "common.h"
#include "int8.h"
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
    if (c.codes) store_int8(y, c.codes, c.absmax, base + k);   // K % 64 == 0: the 8 lanes of a block agree
  }
}

// 8 values as they lie in memory.
template <bool BF16>
struct Raw8 {
  u32x4_t a[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    const char* c = static_cast<const char*>(p) + at * (BF16 ? 2 : 4);
    a[0] = *reinterpret_cast<const u32x4_t*>(c);
    if constexpr (!BF16) a[1] = *reinterpret_cast<const u32x4_t*>(c + 16);
  }
  __device__ __forceinline__ float get(int e) const {
    const u32x4_t& q = a[BF16 ? 0 : e >> 2];
    const uint32_t x[4] = {q.x, q.y, q.z, q.w};
    if constexpr (BF16) return (e & 1) ? __uint_as_float(x[e >> 1] & 0xFFFF0000u) : __uint_as_float(x[e >> 1] << 16);
    else return __uint_as_float(x[e & 3]);
  }
};

// Rows group, group + groups, ...: each group of WAVES waves sums dw over its rows into part[group]. A row's values
// stay in their memory format between the sum and the output (as floats, 6656 bf16 columns took 229 registers, 2
// waves per SIMD).
template <int WAVES, int NV, bool H16, bool W16, bool DW>
__global__ __launch_bounds__(NormShape<WAVES>::kThreads) void norm_bwd_kernel(NormBwd c) {
  using S = NormShape<WAVES>;
  __shared__ float red[16];
  const int t = threadIdx.x % (64 * WAVES);
  const int64_t group = (int64_t)blockIdx.x * S::kRows + threadIdx.x / (64 * WAVES);
  const int64_t groups = (int64_t)gridDim.x * S::kRows;
  float dw[DW ? NV : 1][8];
  if constexpr (DW) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[i][e] = 0.0f;
  }
  for (int64_t row = group; row < c.M; row += groups) {   // uniform for the waves of a row
    const int64_t base = row * c.K;
    Raw8<H16> h[NV], dr[NV];
    Raw8<true> dy[NV];
    Raw8<W16> w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t k = (int64_t)(i * 64 * WAVES + t) * 8;
      if (k >= c.K) continue;
      h[i].load(c.h, base + k);
      dy[i].load(c.dy, base + k);
      if (c.w) w[i].load(c.w, k);
      if (c.dres) dr[i].load(c.dres, base + k);
    }
    const float rstd = c.rstd[row];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t k = (int64_t)(i * 64 * WAVES + t) * 8;
      if (k >= c.K) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = h[i].get(e) * rstd, y = dy[i].get(e);
        if constexpr (DW) dw[i][e] = __builtin_fmaf(y, xh, dw[i][e]);
        sum = __builtin_fmaf(c.w ? y * w[i].get(e) : y, xh, sum);
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
        const float y = dy[i].get(e);
        d[e] = rstd * ((c.w ? y * w[i].get(e) : y) - h[i].get(e) * rstd * mean);
        if (c.dres) d[e] += dr[i].get(e);
      }
      nm_store(c.dh, H16, base + k, d);
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

// dw[k] = the groups' sums, 16 parts of the groups in order (8 loads in flight), then the parts in order. 64 columns
// per workgroup.
__global__ __launch_bounds__(1024) void norm_dw_kernel(const float* __restrict__ part, int groups, int64_t K, float* __restrict__ dw) {
  __shared__ float red[16][64];
  const int c = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int64_t k = (int64_t)blockIdx.x * 64 + c;
  const int per = (groups + 15) / 16, lo = q * per, hi = lo + per < groups ? lo + per : groups;
  float v = 0.0f;
  if (k < K)
    for (int g = lo; g < hi; g += 8) {
      float b[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) b[u] = part[(int64_t)(g + u < hi ? g + u : g) * K + k];
#pragma unroll
      for (int u = 0; u < 8; ++u) v += g + u < hi ? b[u] : 0.0f;
    }
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

// Groups of waves that sum dw: of at least 2 rows where that leaves one per CU (their sums of K floats are written and
// read once more; 1001 x 6656 in groups of 4, 2 and 1 rows 21.6, 19.2 and 25.6 us), at most four per CU.
int norm_slices(int64_t M) {
  const int64_t cus = device_cu_count();
  int64_t n = M / 2;
  if (n < cus) n = M < cus ? M : cus;
  if (n > 4 * cus) n = 4 * cus;
  return (int)(n + 3) / 4 * 4;
}

hipError_t launch_norm_bwd(const NormBwd& c, hipStream_t stream) {
  const int groups = norm_slices(c.M);
  hipError_t e = hipSuccess;
  if (c.M > 0)
    e = by_shape(c.K, [&](auto waves, auto nv) {
      using S = NormShape<decltype(waves)::value>;
      const dim3 grid((unsigned)((groups + S::kRows - 1) / S::kRows));
      auto go = [&](auto h16, auto w16, auto dw) {
        hipLaunchKernelGGL((norm_bwd_kernel<decltype(waves)::value, decltype(nv)::value, decltype(h16)::value,
                                            decltype(w16)::value, decltype(dw)::value>),
                           grid, dim3(S::kThreads), 0, stream, c);
      };
      auto by_w = [&](auto h16, auto dw) { c.w_bf16 ? go(h16, std::true_type{}, dw) : go(h16, std::false_type{}, dw); };
      auto by_h = [&](auto dw) { c.h_bf16 ? by_w(std::true_type{}, dw) : by_w(std::false_type{}, dw); };
      c.dw ? by_h(std::true_type{}) : by_h(std::false_type{});
      return hipGetLastError();
    });
  if (e != hipSuccess || !c.dw) return e;
  hipLaunchKernelGGL(norm_dw_kernel, dim3((unsigned)((c.K + 63) / 64)), dim3(1024), 0, stream, c.part, groups, c.K, c.dw);
  return hipGetLastError();
}

}  // namespace qlora
