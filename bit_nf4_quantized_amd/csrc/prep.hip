// What the products of a layer's pass need beforehand, as one launch of
// independent parts (each workgroup takes a piece of one part): apart, the parts
// of a short batch were mostly launch latency (a linear's backward pass of 200
// rows 101 -> 56 us with this and the joined sums).
//
//   weights   one or two quantised weights [N][K] -> bf16 rows; two of them in
//             pairs of blocks of 32 rows (row n of weight w at 64 (n / 32) + 32 w
//             + n % 32), rows N .. Np zeros. 2.5 B per weight: 90 M weights 45-50 us, 4.5-5.0 TB/s.
//   adapters  32 x 32 tiles, transposed through LDS:
//             l1t [n][rp][K] = L1^T, rows behind the rank zero
//             l2i [2 Np][2 rp] = L2^T in the paired rows' order, weight w's columns
//             at rp w, zeros elsewhere
//             l2p [n][rp][Np] = L2, zeros behind rank and N
//   x         int8 values -> bf16
//   xs        their scales RN32(absmax / 127), [K / 64][M rounded up to 64], zeros behind M
//   dY        [M][N] -> [M][Np], zeros behind N
#include "common.h"
#include "launch.h"

namespace qlora {

namespace {

// DQ: double-quantised constants (decided outside the loop: a branch per unit would wait for each unit's loads).
template <bool DQ>
__device__ __forceinline__ void prep_weights(const LayerPrep& p, const NF4View& W, int which, int block, int blocks,
                                             const float* s_q) {
  const float mu = tensor_mean(W);
  const int64_t K8 = W.cols / 8, nunits = W.rows * K8, all = p.Np * K8;
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(W.codes);
  constexpr int kUnits = 4;                          // 8 weights each, 256 units apart, all loads first
  const int64_t stride = (int64_t)blocks * 256 * kUnits;
  uint32_t c[kUnits];
  float sc[kUnits];
  uint8_t c8[kUnits];
  auto load = [&](int64_t base) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int64_t un = base + (int64_t)u * 256, uc = un < nunits ? un : nunits - 1;
      c[u] = codes[uc];
      const int64_t blk = uc >> 3;
      if constexpr (DQ) c8[u] = W.absmax8[blk];
      sc[u] = DQ ? W.scale2[blk / kDqBlock] : W.absmax32[blk];
    }
  };
  const int64_t first = (int64_t)block * 256 * kUnits + threadIdx.x;
  load(first);
  for (int64_t base = first; base < all; base += stride) {
    uint32_t cc[kUnits];
    float ap[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      cc[u] = c[u];
      ap[u] = DQ ? block_scale(c8[u], sc[u], mu) : sc[u];
    }
    load(base + stride);                             // the next turn's, in flight meanwhile
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int64_t un = base + (int64_t)u * 256;
      if (un >= all) continue;
      const int64_t n = un / K8, k8 = un - n * K8;
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t byte = (cc[u] >> (8 * i)) & 0xFFu;
        o[i] = un < nunits ? pack_bf16x2(s_q[byte & 15u] * ap[u], s_q[byte >> 4] * ap[u]) : 0u;
      }
      const int64_t row = p.n == 2 ? 64 * (n >> 5) + 32 * which + (n & 31) : n;
      *reinterpret_cast<u32x4_t*>(p.wd + row * W.cols + k8 * 8) = u32x4_t{o[0], o[1], o[2], o[3]};
    }
  }
}

__device__ __forceinline__ void prep_l1(const LayerPrep& p, int id, uint16_t (*tile)[33]) {
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, nr = p.rp / 32, per = (int)(p.K / 32) * nr;
  const int which = id / per, i = id - which * per;
  const int64_t k0 = (int64_t)(i / nr) * 32;
  const int j0 = (i % nr) * 32;
  const uint16_t* src = p.L1 + (int64_t)which * p.K * p.r;
  for (int y = ty; y < 32; y += 8) tile[y][tx] = j0 + tx < p.r ? src[(k0 + y) * p.r + j0 + tx] : 0;
  __syncthreads();
  uint16_t* dst = p.l1t + (int64_t)which * p.rp * p.K;
  for (int y = ty; y < 32; y += 8) dst[(int64_t)(j0 + y) * p.K + k0 + tx] = tile[tx][y];
}

__device__ __forceinline__ void prep_l2(const LayerPrep& p, int id, uint16_t (*tile)[33]) {
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, nr = p.rp / 32, per = (int)(p.Np / 32) * nr;
  const int which = id / per, i = id - which * per;
  const int64_t n0 = (int64_t)(i / nr) * 32;
  const int j0 = (i % nr) * 32;
  const uint16_t* src = p.L2 + (int64_t)which * p.r * p.N;
  for (int y = ty; y < 32; y += 8) {
    const uint16_t v = j0 + y < p.r && n0 + tx < p.N ? src[(int64_t)(j0 + y) * p.N + n0 + tx] : 0;
    tile[y][tx] = v;
    if (p.l2p) p.l2p[((int64_t)which * p.rp + j0 + y) * p.Np + n0 + tx] = v;
  }
  if (!p.l2i) return;
  __syncthreads();
  for (int y = ty; y < 32; y += 8) {
    uint16_t* row = p.l2i + (2 * n0 + 32 * which + y) * (2 * p.rp);
    row[which * p.rp + j0 + tx] = tile[tx][y];
    row[(1 - which) * p.rp + j0 + tx] = 0;
  }
}

__global__ __launch_bounds__(256) void layer_prep_kernel(LayerPrep p) {
  __shared__ float s_q[16];
  __shared__ uint16_t tile[32][33];
  __shared__ float scale[64][65];
  int id = (int)blockIdx.x;
  // The weights first where their workgroups take several turns (90 M weights 53 us, last 69: some start late); last
  // where they take one, the others' longer ways beside them (16.8 M weights, 200 rows 14.0 us, first 17.5).
  if (!p.weights_first) id = id + p.blocks[0] < (int)gridDim.x ? id + p.blocks[0] : id + p.blocks[0] - (int)gridDim.x;
  if (id < p.blocks[0]) {
    const int per = p.blocks[0] / p.n;
    const int which = id >= per ? 1 : 0;
    const NF4View W = which ? p.W[1] : p.W[0];
    if (threadIdx.x < 16) s_q[threadIdx.x] = which ? p.tab[1].q[threadIdx.x] : p.tab[0].q[threadIdx.x];
    __syncthreads();
    if (W.absmax32) prep_weights<false>(p, W, which, id - which * per, per, s_q);
    else prep_weights<true>(p, W, which, id - which * per, per, s_q);
    return;
  }
  id -= p.blocks[0];
  if (id < p.blocks[1]) {
    const int64_t n8 = p.M * p.K / 8;
    for (int64_t i = (int64_t)id * 256 + threadIdx.x; i < n8; i += (int64_t)p.blocks[1] * 256) {
      const u32x2_t w = *reinterpret_cast<const u32x2_t*>(p.x8.codes + i * 8);
      const float s = p.x8.absmax[i >> 3] / 127.0f;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (float)(int8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3))) * s;
      *reinterpret_cast<u32x4_t*>(p.x + i * 8) =
          u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    }
    return;
  }
  id -= p.blocks[1];
  if (id < p.blocks[2]) return prep_l1(p, id, tile);
  id -= p.blocks[2];
  if (id < p.blocks[3]) return prep_l2(p, id, tile);
  id -= p.blocks[3];
  if (id < p.blocks[4]) {                            // read by blocks, written by rows, 64 x 64 through LDS
    const int64_t nb = p.K / 64, mp = (p.M + 63) / 64 * 64, mt = mp / 64;
    const int64_t m0 = (id % mt) * 64, b0 = (id / mt) * 64;
    for (int i = threadIdx.x; i < 4096; i += 256) {
      const int64_t m = m0 + (i >> 6), b = b0 + (i & 63);
      scale[i >> 6][i & 63] = m < p.M && b < nb ? p.x8.absmax[m * nb + b] / 127.0f : 0.0f;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 4096; i += 256) {
      const int64_t b = b0 + (i >> 6);
      if (b < nb) p.xs[b * mp + m0 + (i & 63)] = scale[i & 63][i >> 6];
    }
    return;
  }
  id -= p.blocks[4];
  const int64_t per = p.Np / 8, n8 = p.M * per;
  for (int64_t i = (int64_t)id * 256 + threadIdx.x; i < n8; i += (int64_t)p.blocks[5] * 256) {
    const int64_t m = i / per, c = (i - m * per) * 8;   // N % 8 == 0
    u32x4_t v = {0u, 0u, 0u, 0u};
    if (c < p.N) v = *reinterpret_cast<const u32x4_t*>(p.dy + m * p.N + c);
    *reinterpret_cast<u32x4_t*>(p.dyp + m * p.Np + c) = v;
  }
}

}  // namespace

hipError_t launch_layer_prep(LayerPrep p, hipStream_t stream) {
  const int64_t cus = device_cu_count();
  auto blocks = [&](int64_t units, int64_t most) {
    const int64_t b = (units + 255) / 256;
    return (int)(b < most ? b : most);
  };
  p.blocks[0] = p.wd ? p.n * blocks(p.Np * p.K / 32, 8 * cus / p.n) : 0;
  p.weights_first = p.n * p.Np * p.K / 8 > (int64_t)p.blocks[0] * 1024;   // 1024: a workgroup's units per turn
  p.blocks[1] = p.x ? blocks(p.M * p.K / 8, 8 * cus) : 0;
  p.blocks[2] = p.l1t ? p.n * (int)(p.K / 32) * (p.rp / 32) : 0;
  p.blocks[3] = p.l2i || p.l2p ? p.n * (int)(p.Np / 32) * (p.rp / 32) : 0;
  p.blocks[4] = p.xs ? (int)((p.M + 63) / 64 * ((p.K / 64 + 63) / 64)) : 0;
  p.blocks[5] = p.dyp ? blocks(p.M * p.Np / 8, 8 * cus) : 0;
  int64_t all = 0;
  for (int b : p.blocks) all += b;
  if (all == 0) return hipSuccess;
  hipLaunchKernelGGL(layer_prep_kernel, dim3((unsigned)all), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace qlora
