// The dequantisers that feed the dense GEMM, as workgroup bodies (256 threads):
// kernels of their own (dense_gemm.hip), or beside other work in one launch
// (multi.hip).
#pragma once

#include "common.h"
#include "launch.h"

namespace qlora {

// Wd[n][k] for the forward product, the standalone dequant arithmetic
// (bf16(RN32(q[code] * a'))). A thread takes 4 units of 8 weights (one code
// dword, one 16-byte store) 256 units apart, so that every load and store
// instruction of a wave covers one contiguous range; the 4 code loads and
// block constants are issued before any store (measured 17.0 us against
// 19.5 us per launch for one unit of 16 weights per thread).
constexpr int kRowsUnits = 4;
__device__ __forceinline__ void dequant_rows_body(const NF4View& W, const NF4Table& tab, uint16_t* __restrict__ out,
                                                  int block, int blocks) {
  __shared__ float s_q[16];
  if (threadIdx.x < 16) s_q[threadIdx.x] = tab.q[threadIdx.x];
  __syncthreads();
  const float mu = tensor_mean(W);
  const int64_t nunits = W.rows * W.cols / 8;  // cols % 64 == 0
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(W.codes);
  const int64_t stride = (int64_t)blocks * 256 * kRowsUnits;
  for (int64_t base = (int64_t)block * 256 * kRowsUnits + threadIdx.x; base < nunits; base += stride) {
    uint32_t c[kRowsUnits];
    float ap[kRowsUnits];
#pragma unroll
    for (int u = 0; u < kRowsUnits; ++u) {
      const int64_t un = base + (int64_t)u * 256;
      const int64_t uc = un < nunits ? un : nunits - 1;  // clamped: loads stay unconditional
      c[u] = codes[uc];
      ap[u] = block_const(W, uc >> 3, mu);  // 8 units per 64-block
    }
#pragma unroll
    for (int u = 0; u < kRowsUnits; ++u) {
      const int64_t un = base + (int64_t)u * 256;
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t byte = (c[u] >> (8 * i)) & 0xFFu;
        o[i] = pack_bf16x2(s_q[byte & 15u] * ap[u], s_q[byte >> 4] * ap[u]);
      }
      if (un < nunits) *reinterpret_cast<u32x4_t*>(out + un * 8) = u32x4_t{o[0], o[1], o[2], o[3]};
    }
  }
}

// WdT[k][n] = Wd[n][k] for the dX product, rows padded to ldo >= N columns
// with zeros, without LDS: a thread dequantises two adjacent weight rows
// (n, n+1) over 32 k (16 code bytes each, inside one 64-block), so that each
// (row n, row n+1) pair at one k is one dword of output row k; the 64 lanes
// of a wave take 64 consecutive row pairs, so every store instruction
// writes 256 contiguous bytes. Workgroup: 128 rows n x 128 k (4 waves along k).
__device__ __forceinline__ void dequant_cols_body(const NF4View& W, const NF4Table& tab, uint16_t* __restrict__ out,
                                                  int64_t ldo, int bx, int by) {
  __shared__ float s_q[16];
  if (threadIdx.x < 16) s_q[threadIdx.x] = tab.q[threadIdx.x];
  __syncthreads();
  const float mu = tensor_mean(W);
  const int64_t K = W.cols, N = W.rows;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t n = (int64_t)by * 128 + 2 * lane;           // rows n, n + 1 (N % 8 == 0)
  const int64_t k0 = (int64_t)bx * 128 + wave * 32;         // k0 .. k0 + 32
  if (k0 >= K) return;                                              // wave-uniform; no barrier follows
  const bool in = n < N;
  const int64_t na = in ? n : 0;
  const int64_t e0 = na * K + k0, e1 = e0 + K;
  const u32x4_t ca = *reinterpret_cast<const u32x4_t*>(W.codes + (e0 >> 1));
  const u32x4_t cb = *reinterpret_cast<const u32x4_t*>(W.codes + (e1 >> 1));
  const float aa = block_const(W, e0 / kBlock, mu), ab = block_const(W, e1 / kBlock, mu);
  const uint32_t wa[4] = {ca.x, ca.y, ca.z, ca.w}, wb[4] = {cb.x, cb.y, cb.z, cb.w};
  if (n >= ldo) return;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const uint32_t qa = (wa[i >> 3] >> (4 * (i & 7))) & 15u;
    const uint32_t qb = (wb[i >> 3] >> (4 * (i & 7))) & 15u;
    const uint32_t v = in ? pack_bf16x2(s_q[qa] * aa, s_q[qb] * ab) : 0u;
    *reinterpret_cast<uint32_t*>(out + (k0 + i) * ldo + n) = v;
  }
}

// Workgroups of the two: rows (grid-stride), and columns x rows of 128 x 128.
inline int64_t dequant_rows_blocks(const NF4View& W) {
  const int64_t per_block = 256 * kRowsUnits;
  const int64_t blocks = (W.rows * W.cols / 8 + per_block - 1) / per_block;
  const int64_t cap = (int64_t)device_cu_count() * 8;
  return blocks < cap ? blocks : cap;
}

}  // namespace qlora
