// The gated feed-forward block over two quantised bases with adapters, for
// gfx950:
//
//   G = X Wg^T + s (X L1g) L2g,   U = X Wu^T + s (X L1u) L2u,   A = act(G) U
//   dU = dA act(G),  dG = dA U act'(G)
//   dX = dG Wg + dU Wu + s (dG L2g^T) L1g^T + s (dU L2u^T) L1u^T,  dL1, dL2 as for the linear
//
// with act(g) = g sigma(z): z = g (SiLU) or z = sqrt(8 / pi) (g + 0.044715 g^3)
// (GELU in its tanh form), act'(g) = sigma + g sigma (1 - sigma) dz/dg.
//
// Both weights are dequantised into one matrix [2 Fp][K] (Fp: F rounded up to
// 64) whose rows alternate in blocks of 32, gate and up, so that the 64 columns
// of a GEMM wave hold G and U of the same 32 features in the same lanes and
// registers: the product act(G) U is made from the accumulators, and only A is
// written. The backward pass without kept activations runs the same product,
// with an epilogue that reads dA and writes dG and dU; with G and U kept in 8
// bits an elementwise kernel makes them. dX is one product over both, [dG dU]
// against the same matrix read down its rows.
//
// Bound by the matrix units where rows are many, in long runs of calls, 4096 -> 2 x 11008: dX of 8192 rows 1096-1107 us
// (1.35 PFLOP/s; a large library product 1.46), the product computed again for the backward pass 1187-1202 (1.27); the
// forward product of 2048 rows 290 us, with 8-bit stores 306-311 (1.24: 688 tiles are 2.7 rounds of the CUs); 391 rows
// 100 (172 tiles on 256 CUs). dG and dU from 8 bits, 8192 rows, 138 us (5.3 TB/s). The adapters' second products are the
// last stages of the same tiles (a slab of 2 rp columns, beside K or 2 Fp of the base).
#include "act.h"
#include "common.h"
#include "int8.h"
#include "launch.h"
#include "tile_gemm.h"

namespace qlora {

namespace {

int64_t gd_cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---- the product with its epilogues ------------------------------------------------------

// Epilogue tile in LDS: one 32-row block of every wave at a time, gate and up as fp32, 64 rows (both wave rows) x 128
// features; the threads then take 8 features of a row each.
constexpr int kEpPitch = 128 + 4;

struct GatedOut {
  uint16_t* A;
  int8_t* codes[2];    // gate, up; nullptr: not kept
  float* absmax[2];
  int64_t M, F;
};

// A = act(G) U, and the 8-bit values of G and U.
template <int ACT, bool SAVE>
struct GatedFwdEpi {
  GatedOut o;
  template <int MI>
  __device__ __forceinline__ void operator()(f32x16_t (&acc)[MI][2], int64_t m0, int64_t n0, int wm, int wn, int z,
                                             uint16_t* smem) const {
    const int lane = threadIdx.x & 63, tid = threadIdx.x;
    const int64_t f0 = n0 / 2;
    if constexpr (!SAVE) {
      // a wave's 32 rows x 32 features as bf16 in its own padded LDS slice, then 16-byte stores
      constexpr int kPitch = 32 + 8;
      uint16_t* ep = smem + (wm * 4 + wn) * (32 * kPitch);
#pragma unroll
      for (int i = 0; i < MI; ++i) {
#pragma unroll
        for (int v = 0; v < 16; ++v)
          ep[((v & 3) + 4 * (lane >> 5) + 8 * (v >> 2)) * kPitch + (lane & 31)] =
              f32_to_bf16(act_of<ACT>(acc[i][0][v]) * acc[i][1][v]);
        __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave's writes to its own slice
#pragma unroll
        for (int it = 0; it < 2; ++it) {
          const int r = 16 * it + (lane >> 2), c = 8 * (lane & 3);
          const u32x4_t val = *reinterpret_cast<const u32x4_t*>(ep + r * kPitch + c);
          const int64_t row = m0 + (wm * MI + i) * 32 + r, f = f0 + 32 * wn + c;
          if (row < o.M && f < o.F) *reinterpret_cast<u32x4_t*>(o.A + row * o.F + f) = val;
        }
        __builtin_amdgcn_s_waitcnt(0xc07f);
      }
    } else {
      float* eg = reinterpret_cast<float*>(smem);
      float* eu = eg + 64 * kEpPitch;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        if (i > 0) __syncthreads();
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int at = (32 * wm + (v & 3) + 4 * (lane >> 5) + 8 * (v >> 2)) * kEpPitch + 32 * wn + (lane & 31);
          eg[at] = acc[i][0][v];
          eu[at] = acc[i][1][v];
        }
        __syncthreads();
#pragma unroll
        for (int it = 0; it < 2; ++it) {
          const int rl = 32 * it + (tid >> 4), c = 8 * (tid & 15);
          const int64_t row = m0 + ((rl >> 5) * MI + i) * 32 + (rl & 31), f = f0 + c;
          float g[8], u[8], a[8];
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            const f32x4_t gv = *reinterpret_cast<const f32x4_t*>(eg + rl * kEpPitch + c + e);
            const f32x4_t uv = *reinterpret_cast<const f32x4_t*>(eu + rl * kEpPitch + c + e);
            g[e] = gv.x; g[e + 1] = gv.y; g[e + 2] = gv.z; g[e + 3] = gv.w;
            u[e] = uv.x; u[e + 1] = uv.y; u[e + 2] = uv.z; u[e + 3] = uv.w;
          }
          if (row < o.M && f < o.F) {     // F % 64 == 0: the 8 lanes of a block agree
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] = act_of<ACT>(g[e]) * u[e];
            const int64_t at = row * o.F + f;
            *reinterpret_cast<u32x4_t*>(o.A + at) = u32x4_t{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                                                            pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7])};
            store_int8(g, o.codes[0], o.absmax[0], at);
            store_int8(u, o.codes[1], o.absmax[1], at);
          }
        }
      }
    }
  }
};

// dG = dA U act'(G), dU = dA act(G) of the recomputed G and U, rounded to bf16 once: they are the operands of the
// products that follow.
template <int ACT>
struct GatedBwdEpi {
  const uint16_t* dA;
  uint16_t* dgu;         // [M][2 Fp]
  int64_t M, F, Fp;
  template <int MI>
  __device__ __forceinline__ void operator()(f32x16_t (&acc)[MI][2], int64_t m0, int64_t n0, int wm, int wn, int z,
                                             uint16_t* smem) const {
    const int lane = threadIdx.x & 63;
    const int64_t f0 = n0 / 2 + 32 * wn;
    constexpr int kPitch = 32 + 8;
    uint16_t* eg = smem + (wm * 4 + wn) * (2 * 32 * kPitch);
    uint16_t* eu = eg + 32 * kPitch;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int64_t row0 = m0 + (wm * MI + i) * 32;
#pragma unroll
      for (int it = 0; it < 2; ++it) {          // dA through the slice
        const int r = 16 * it + (lane >> 2), c = 8 * (lane & 3);
        const bool in = row0 + r < M && f0 + c < F;
        u32x4_t val = {0u, 0u, 0u, 0u};
        if (in) val = *reinterpret_cast<const u32x4_t*>(dA + (row0 + r) * F + f0 + c);
        *reinterpret_cast<u32x4_t*>(eg + r * kPitch + c) = val;
      }
      __builtin_amdgcn_s_waitcnt(0xc07f);
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int at = ((v & 3) + 4 * (lane >> 5) + 8 * (v >> 2)) * kPitch + (lane & 31);
        const float d = bf16_to_f32(eg[at]);
        float a, da;
        act_both<ACT>(acc[i][0][v], &a, &da);
        // columns from F on: dA and the weights' padding are zeros
        eg[at] = f32_to_bf16(d * acc[i][1][v] * da);
        eu[at] = f32_to_bf16(d * a);
      }
      __builtin_amdgcn_s_waitcnt(0xc07f);
#pragma unroll
      for (int it = 0; it < 2; ++it) {
        const int r = 16 * it + (lane >> 2), c = 8 * (lane & 3);
        const int64_t row = row0 + r, f = f0 + c;
        if (row < M && f < Fp) {
          *reinterpret_cast<u32x4_t*>(dgu + row * (2 * Fp) + f) = *reinterpret_cast<const u32x4_t*>(eg + r * kPitch + c);
          *reinterpret_cast<u32x4_t*>(dgu + row * (2 * Fp) + Fp + f) = *reinterpret_cast<const u32x4_t*>(eu + r * kPitch + c);
        }
      }
      __builtin_amdgcn_s_waitcnt(0xc07f);
    }
  }
};

// bf16 output, dense [M][N]; or, in reduction slices, fp32 partials [slices][M][N].
struct StoreEpi {
  uint16_t* C;
  float* part;
  int64_t M, N;
  template <int MI>
  __device__ __forceinline__ void operator()(f32x16_t (&acc)[MI][2], int64_t m0, int64_t n0, int wm, int wn, int z,
                                             uint16_t* smem) const {
    const int lane = threadIdx.x & 63;
    if (part) {
      tg_store_partial(acc, part + (int64_t)z * M * N, M, N, m0, n0, wm, wn);
      return;
    }
    constexpr int kPitch = 64 + 8;
    uint16_t* ep = smem + (wm * 4 + wn) * (32 * kPitch);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v)
          ep[((v & 3) + 4 * (lane >> 5) + 8 * (v >> 2)) * kPitch + 32 * j + (lane & 31)] = f32_to_bf16(acc[i][j][v]);
      __builtin_amdgcn_s_waitcnt(0xc07f);
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int r = 8 * it + (lane >> 3), c = 8 * (lane & 7);
        const u32x4_t val = *reinterpret_cast<const u32x4_t*>(ep + r * kPitch + c);
        const int64_t row = m0 + (wm * MI + i) * 32 + r, col = n0 + 64 * wn + c;
        if (row < M && col < N) *reinterpret_cast<u32x4_t*>(C + row * N + col) = val;
      }
      __builtin_amdgcn_s_waitcnt(0xc07f);
    }
  }
};

template <class L, class E>
__global__ __launch_bounds__(kTgThreads, 1) void gated_gemm_kernel(TgArgs p, E epi, TgPlan pl) {
  __shared__ __attribute__((aligned(1024))) uint16_t smem[kTgSmem];
  tg_run<L>(p, epi, pl, smem);
}

template <class L, class E>
hipError_t run_tiles(const TgArgs& p, const E& epi, const TgPlan& pl, hipStream_t stream) {
  hipLaunchKernelGGL((gated_gemm_kernel<L, E>), dim3((unsigned)(pl.tiles_m * pl.tiles_n * pl.slices)), dim3(kTgThreads), 0, stream,
                     p, epi, pl);
  return hipGetLastError();
}

using RowRow = TgLayout<false, false, true, false>;
using RowPaired = TgLayout<false, true, true, true>;
using RowDown = TgLayout<false, true, true, false>;

// ---- elementwise parts -----------------------------------------------------------------------

__device__ __forceinline__ void load_int8(const int8_t* codes, const float* absmax, int64_t at, float* v) {
  const u32x2_t w = *reinterpret_cast<const u32x2_t*>(codes + at);
  const float s = absmax[at >> 6] / 127.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (float)(int8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3))) * s;
}

__device__ __forceinline__ void load_bf16(const uint16_t* p, float* v) {
  const u32x4_t w = *reinterpret_cast<const u32x4_t*>(p);
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __uint_as_float(x[e] << 16);
    v[2 * e + 1] = __uint_as_float(x[e] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ u32x4_t pack8(const float* v) {
  return u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

// dG and dU from the kept 8-bit G and U (F a multiple of 64), 8 features per thread.
template <int ACT>
__global__ __launch_bounds__(256) void gated_dgu_kernel(const uint16_t* __restrict__ dA, Int8Values G, Int8Values U,
                                                        int64_t M, int64_t F, uint16_t* __restrict__ dgu) {
  const int64_t n = M * F / 8, per = F / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per, f = (i - row * per) * 8;
    float g[8], u[8], d[8], dg[8], du[8];
    load_int8(G.codes, G.absmax, i * 8, g);
    load_int8(U.codes, U.absmax, i * 8, u);
    load_bf16(dA + i * 8, d);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float a, da;
      act_both<ACT>(g[e], &a, &da);
      dg[e] = d[e] * u[e] * da;
      du[e] = d[e] * a;
    }
    *reinterpret_cast<u32x4_t*>(dgu + row * 2 * F + f) = pack8(dg);
    *reinterpret_cast<u32x4_t*>(dgu + row * 2 * F + F + f) = pack8(du);
  }
}

// ---- few rows ------------------------------------------------------------------------------------

// A (and the 8-bit values) from the base products' partials [S][M][F] of each weight and the adapters' T partials
// [2][Z][M][r]: 16 rows and 128 features per workgroup, one row and 8 features per thread. The adapters' second factors
// come through LDS in pieces of 64 ranks (all loads of a piece in flight; read rank by rank from memory, one token of
// rank 64 took 39 us here). Slices and ranks are added in order.
constexpr int kFinRanks = 64;

template <int ACT>
__global__ __launch_bounds__(256) void gated_finish_kernel(const float* __restrict__ part, int S,
                                                           const float* __restrict__ tpart, int Z, int r, float s,
                                                           const uint16_t* __restrict__ L2, uint16_t* __restrict__ T_out,
                                                           GatedOut o) {
  __shared__ float sT[2][16][kFinRanks + 4];
  __shared__ __attribute__((aligned(16))) uint16_t sL[2][kFinRanks][128];
  const int tid = threadIdx.x, lr = tid >> 4;
  const int64_t f0 = (int64_t)blockIdx.x * 128, f = f0 + 8 * (tid & 15);
  const int64_t row0 = (int64_t)blockIdx.y * 16, row = row0 + lr;
  const bool in = row < o.M && f < o.F;
  const int64_t at = in ? row * o.F + f : 0, all = o.M * o.F;
  const int rows = (int)(o.M - row0 < 16 ? o.M - row0 : 16);
  float v[2][8] = {};
  constexpr int kSlices = 4;                       // that many slices' loads in flight
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const float* p = part + (int64_t)w * S * all + at;
    for (int z = 0; z < S; z += kSlices) {
      f32x4_t a[kSlices], b[kSlices];
#pragma unroll
      for (int u = 0; u < kSlices; ++u) {
        const float* q = p + (z + u < S ? z + u : z) * all;
        a[u] = *reinterpret_cast<const f32x4_t*>(q);
        b[u] = *reinterpret_cast<const f32x4_t*>(q + 4);
      }
#pragma unroll
      for (int u = 0; u < kSlices; ++u) {
        if (z + u >= S) break;                     // uniform
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[w][e] += a[u][e];
          v[w][4 + e] += b[u][e];
        }
      }
    }
  }
  for (int j0 = 0; j0 < r; j0 += kFinRanks) {
    const int n = r - j0 < kFinRanks ? r - j0 : kFinRanks;      // a multiple of 8
    if (j0 > 0) __syncthreads();
    // L2 [2][n][128 features]: 16 chunks of 16 bytes per rank
#pragma unroll
    for (int i = 0; i < 2 * kFinRanks * 16 / 256; ++i) {
      const int c = tid + 256 * i, w = c / (kFinRanks * 16), j = c / 16 % kFinRanks, ch = c % 16;
      if (j < n && f0 + 8 * ch < o.F)
        *reinterpret_cast<u32x4_t*>(&sL[w][j][8 * ch]) =
            *reinterpret_cast<const u32x4_t*>(L2 + ((int64_t)w * r + j0 + j) * o.F + f0 + 8 * ch);
    }
    for (int i = tid; i < 2 * rows * n; i += 256) {
      const int w = i / (rows * n), k = i / n % rows, j = i % n;
      const float* p = tpart + (((int64_t)w * Z) * o.M + row0 + k) * r + j0 + j;
      float t = 0.0f;
      for (int z = 0; z < Z; z += 8) {             // loads of 8 slices in flight, added in order
        float b[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) b[u] = p[(int64_t)(z + u < Z ? z + u : z) * o.M * r];
#pragma unroll
        for (int u = 0; u < 8; ++u) t += z + u < Z ? b[u] : 0.0f;
      }
      sT[w][k][j] = bf16_to_f32(f32_to_bf16(s * t));
      if (T_out && blockIdx.x == 0) T_out[((int64_t)w * o.M + row0 + k) * r + j0 + j] = f32_to_bf16(t);
    }
    __syncthreads();
    if (in) {
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
          const float x = sT[w][lr][j];
          float y[8];
          load_bf16(&sL[w][j][8 * (tid & 15)], y);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[w][e] = __builtin_fmaf(x, y[e], v[w][e]);
        }
    }
  }
  if (!in) return;
  float a[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) a[e] = act_of<ACT>(v[0][e]) * v[1][e];
  *reinterpret_cast<u32x4_t*>(o.A + at) = pack8(a);
  if (o.codes[0]) {                                // F % 64 == 0: whole blocks per 8 lanes
    store_int8(v[0], o.codes[0], o.absmax[0], at);
    store_int8(v[1], o.codes[1], o.absmax[1], at);
  }
}

}  // namespace

namespace {

TgPlan dx_plan(int64_t M, int64_t K, int64_t reduction) {
  return tg_plan(M, K, (int)(reduction / kTgK), tg_partial_rows(M), device_cu_count());
}

}  // namespace

LayerWorkspace gated_workspace_layout(int64_t M, int64_t K, int64_t F, int r, bool bwd) {
  const int64_t Fp = gd_cdiv(F, 64) * 64, rp = gd_cdiv(r, 64) * 64;
  LayerWorkspace L;
  size_t off = 0;
  auto take = [&](int64_t bytes) { const size_t at = off; off += align_up((size_t)bytes, 256); return at; };
  const bool dense = bwd || M > kMultiSmallRows;
  L.wd_off = take(dense ? 2 * Fp * K * 2 : 0);
  L.l1t_off = take(dense ? 2 * rp * K * 2 : 0);
  L.l2i_off = take(dense ? (2 * Fp) * (2 * rp) * 2 : 0);
  L.l2p_off = take(bwd ? 2 * rp * Fp * 2 : 0);
  L.st_off = take(M * 2 * rp * 2);
  L.t_off = take(bwd ? 2 * M * r * 2 : 0);
  L.dy_off = take(bwd ? M * 2 * Fp * 2 : 0);
  L.x_off = take(bwd ? M * K * 2 : 0);
  L.xs_off = take(bwd ? gd_cdiv(M, 64) * K * 4 : 0);
  int64_t part = (int64_t)adapter_partial_bytes(AdapterShape{2, M, K, Fp, r, 0.0f});
  if (2 * (int64_t)gemv1_partial_bytes(K, r) > part) part = 2 * gemv1_partial_bytes(K, r);
  L.part_off = take(part);
  const int64_t few = M < kMultiSmallRows ? M : kMultiSmallRows;
  L.part2_off = take(bwd ? tg_partial_rows(M) * K * 4 : small_pair_partial_floats(few, K, F) * 4);
  L.total = off > 0 ? off : 256;
  return L;
}

LayerWorkspace linear_int8_workspace_layout(int64_t M, int64_t K, int64_t N, int r) {
  const int64_t Np = gd_cdiv(N, 64) * 64, rp = gd_cdiv(r, 64) * 64;
  LayerWorkspace L;
  size_t off = 0;
  auto take = [&](int64_t bytes) { const size_t at = off; off += align_up((size_t)bytes, 256); return at; };
  L.wd_off = take(Np * K * 2);
  L.l1t_off = take(rp * K * 2);
  L.l2i_off = off;
  L.l2p_off = take(rp * Np * 2);
  L.st_off = take(M * rp * 2);
  L.t_off = take(M * r * 2);
  L.dy_off = take(Np != N ? M * Np * 2 : 0);
  L.x_off = take(M * K * 2);
  L.xs_off = take(gd_cdiv(M, 64) * K * 4);
  L.part_off = take((int64_t)adapter_partial_bytes(AdapterShape{1, M, K, Np, r, 0.0f}));
  L.part2_off = take(tg_partial_rows(M) * K * 4);
  L.total = off > 0 ? off : 256;
  return L;
}

namespace {

struct LayerBuffers {
  uint16_t *wd, *l1t, *l2i, *l2p, *st, *t, *dy, *x;
  float *xs, *part, *part2;
  LayerBuffers(const LayerWorkspace& L, void* ws) {
    char* b = static_cast<char*>(ws);
    auto at = [&](size_t off) { return reinterpret_cast<uint16_t*>(b + off); };
    wd = at(L.wd_off);
    l1t = at(L.l1t_off);
    l2i = at(L.l2i_off);
    l2p = at(L.l2p_off);
    st = at(L.st_off);
    t = at(L.t_off);
    dy = at(L.dy_off);
    x = at(L.x_off);
    xs = reinterpret_cast<float*>(b + L.xs_off);
    part = reinterpret_cast<float*>(b + L.part_off);
    part2 = reinterpret_cast<float*>(b + L.part2_off);
  }
};

LayerPrep gated_prep(const GatedBase& W, int64_t M, const uint16_t* L1, const uint16_t* L2, int r) {
  LayerPrep p{};
  p.n = 2;
  p.M = M;
  p.K = W.gate.cols;
  p.N = W.gate.rows;
  p.Np = gd_cdiv(p.N, 64) * 64;
  p.r = r;
  p.rp = (int)gd_cdiv(r, 64) * 64;
  p.W[0] = W.gate;
  p.W[1] = W.up;
  p.tab[0] = W.tab_gate;
  p.tab[1] = W.tab_up;
  p.L1 = L1;
  p.L2 = L2;
  return p;
}

// X as int8 values: dL1 reads them as they are (rank <= 64), the other products of X a bf16 copy.
void lay_int8(LayerPrep& p, const LayerBuffers& b, const Int8Values& x8, bool products) {
  p.x8 = x8;
  p.xs = p.r <= 64 ? b.xs : nullptr;
  p.x = products || p.r > 64 ? b.x : nullptr;
}

// The product of X with both weights and their adapters, into `epi`.
template <class E>
hipError_t gated_product(const LayerBuffers& b, const uint16_t* X, const LayerPrep& s, const E& epi, hipStream_t stream) {
  TgArgs p{};
  p.A = {X, s.K, s.M};
  p.B = {b.wd, s.K, 2 * s.Np};
  p.A2 = {b.st, 2 * s.rp, s.M};
  p.B2 = {b.l2i, 2 * s.rp, 2 * s.Np};
  p.kmain = s.K;
  p.kslab = 2 * s.rp;
  return run_tiles<RowRow>(p, epi, tg_plan(s.M, 2 * s.Np, (int)((p.kmain + p.kslab) / kTgK), 0, device_cu_count()), stream);
}

template <typename F1, typename F2>
hipError_t by_act(int act, F1&& silu, F2&& gelu) { return act == kActSilu ? silu() : gelu(); }

#define GD_TRY(call)                       \
  do {                                     \
    const hipError_t e_ = (call);          \
    if (e_ != hipSuccess) return e_;       \
  } while (0)

// dX (unless NULL), dL1 and dL2 of s.n linears of one input from their upstream gradients, side by side in rows of
// n Np: s U (and T_out, where T is not there yet), dX with the weights read down their rows, the adapters' gradients
// beside the sums of dX's slices.
template <class L>
hipError_t layer_grads(const LayerPrep& s, const LayerBuffers& b, const uint16_t* X, const int8_t* x8, const uint16_t* dY, float scale,
                       const uint16_t* T, bool have_t, uint16_t* dX, void* dL1, void* dL2, bool grad_bf16,
                       hipStream_t stream) {
  const int64_t ldy = s.n * s.Np;
  const AdapterShape sh{s.n, s.M, s.K, s.N, s.r, scale};
  const AdapterOperands o{X, x8, b.xs, s.L1, b.l1t, dY, ldy, s.Np, b.l2p, s.Np};
  GD_TRY(adapter_up(sh, o, b.st, have_t ? nullptr : b.t, b.part, stream));
  SplitSum sum{b.part2, dX, s.M * s.K, 1};
  if (dX) {
    TgArgs p{};
    p.A = {dY, ldy, s.M};
    p.B = {b.wd, s.K, s.K};
    p.A2 = {b.st, s.n * s.rp, s.M};
    p.B2 = {b.l1t, s.K, s.K};
    p.kmain = ldy;
    p.kslab = s.n * s.rp;
    p.krows_b = ldy;
    const TgPlan pl = dx_plan(s.M, s.K, p.kmain + p.kslab);
    sum.S = pl.slices;
    GD_TRY(run_tiles<L>(p, StoreEpi{dX, pl.slices > 1 ? b.part2 : nullptr, s.M, s.K}, pl, stream));
  }
  return adapter_grads(sh, o, b.st, have_t ? T : b.t, dL1, dL2, grad_bf16, b.part, dX && sum.S > 1 ? &sum : nullptr, stream);
}

__global__ __launch_bounds__(256) void zero_kernel(uint32_t* __restrict__ p, int64_t words) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words; i += (int64_t)gridDim.x * 256) p[i] = 0u;
}

// The gradients of an empty batch (a fill kernel: the call may be captured).
hipError_t zero_grads(int64_t n1, int64_t n2, void* dL1, void* dL2, bool grad_bf16, hipStream_t stream) {
  const int64_t per = grad_bf16 ? 2 : 1;             // values per word; both counts are multiples of 8
  hipLaunchKernelGGL(zero_kernel, dim3(256), dim3(256), 0, stream, static_cast<uint32_t*>(dL1), n1 / per);
  hipLaunchKernelGGL(zero_kernel, dim3(256), dim3(256), 0, stream, static_cast<uint32_t*>(dL2), n2 / per);
  return hipGetLastError();
}

}  // namespace

hipError_t gated_forward(const GatedBase& W, const uint16_t* X, int64_t M, const uint16_t* L1, const uint16_t* L2, int r,
                         float s, int act, uint16_t* A, uint16_t* T_out, const Int8Values* gate8, const Int8Values* up8,
                         void* ws, hipStream_t stream) {
  const int64_t K = W.gate.cols, F = W.gate.rows;
  if (M == 0) return hipSuccess;
  const LayerBuffers b(gated_workspace_layout(M, K, F, r, false), ws);
  GatedOut o{A, {gate8 ? gate8->codes : nullptr, up8 ? up8->codes : nullptr},
             {gate8 ? gate8->absmax : nullptr, up8 ? up8->absmax : nullptr}, M, F};
  if (!gate8 && gemv1_pair_applies(W, M, r)) return launch_gemv1_pair(W, X, L1, L2, r, s, act, A, T_out, b.part, stream);
  if (M <= kMultiSmallRows) {      // one pass over the 4-bit weights
    GD_TRY(launch_small_pair(W, X, M, L1, r, b.part, b.part2, stream));
    const int S = small_pair_slices(M, K, F), Z = small_t_slices(K);
    const dim3 grid((unsigned)gd_cdiv(F, 128), (unsigned)gd_cdiv(M, 16));
    if (act == kActSilu)
      hipLaunchKernelGGL(gated_finish_kernel<kActSilu>, grid, dim3(256), 0, stream, b.part2, S, b.part, Z, r, s, L2, T_out, o);
    else
      hipLaunchKernelGGL(gated_finish_kernel<kActGelu>, grid, dim3(256), 0, stream, b.part2, S, b.part, Z, r, s, L2, T_out, o);
    return hipGetLastError();
  }
  LayerPrep p = gated_prep(W, M, L1, L2, r);
  p.wd = b.wd;
  p.l1t = b.l1t;
  p.l2i = b.l2i;
  GD_TRY(launch_layer_prep(p, stream));
  GD_TRY(adapter_down(AdapterShape{2, M, K, F, r, s}, AdapterOperands{X, nullptr, nullptr, L1, b.l1t, nullptr, 0, 0, nullptr, 0}, b.st, T_out,
                      b.part, stream));
  if (gate8)
    return by_act(
        act, [&] { return gated_product(b, X, p, GatedFwdEpi<kActSilu, true>{o}, stream); },
        [&] { return gated_product(b, X, p, GatedFwdEpi<kActGelu, true>{o}, stream); });
  return by_act(
      act, [&] { return gated_product(b, X, p, GatedFwdEpi<kActSilu, false>{o}, stream); },
      [&] { return gated_product(b, X, p, GatedFwdEpi<kActGelu, false>{o}, stream); });
}

hipError_t gated_backward(const GatedBase& W, const uint16_t* X, const Int8Values* X8, const uint16_t* dA, int64_t M,
                          const uint16_t* L1, const uint16_t* L2, int r, float s, int act, const uint16_t* T,
                          const Int8Values* gate8, const Int8Values* up8, uint16_t* dX, void* dL1, void* dL2,
                          bool grad_bf16, void* ws, hipStream_t stream) {
  const int64_t K = W.gate.cols, F = W.gate.rows;
  if (M == 0) return zero_grads(2 * K * r, 2 * r * F, dL1, dL2, grad_bf16, stream);
  const LayerBuffers b(gated_workspace_layout(M, K, F, r, true), ws);
  LayerPrep p = gated_prep(W, M, L1, L2, r);
  p.wd = !gate8 || dX ? b.wd : nullptr;
  p.l1t = b.l1t;
  p.l2i = gate8 ? nullptr : b.l2i;
  p.l2p = b.l2p;
  if (X8) {
    lay_int8(p, b, *X8, !gate8 || !T);
    X = b.x;
  }
  GD_TRY(launch_layer_prep(p, stream));
  bool have_t = T != nullptr;
  if (!gate8) {
    GD_TRY(adapter_down(AdapterShape{2, M, K, F, r, s}, AdapterOperands{X, nullptr, nullptr, L1, b.l1t, nullptr, 0, 0, nullptr, 0}, b.st,
                        T ? nullptr : b.t, b.part, stream));
    GD_TRY(by_act(
        act, [&] { return gated_product(b, X, p, GatedBwdEpi<kActSilu>{dA, b.dy, M, F, p.Np}, stream); },
        [&] { return gated_product(b, X, p, GatedBwdEpi<kActGelu>{dA, b.dy, M, F, p.Np}, stream); }));
    if (!have_t) {
      T = b.t;
      have_t = true;
    }
  } else {
    int64_t blocks = gd_cdiv(M * F / 8, 256);
    if (blocks > 16 * device_cu_count()) blocks = 16 * device_cu_count();
    if (act == kActSilu)
      hipLaunchKernelGGL(gated_dgu_kernel<kActSilu>, dim3((unsigned)blocks), dim3(256), 0, stream, dA, *gate8, *up8, M, F, b.dy);
    else
      hipLaunchKernelGGL(gated_dgu_kernel<kActGelu>, dim3((unsigned)blocks), dim3(256), 0, stream, dA, *gate8, *up8, M, F, b.dy);
    GD_TRY(hipGetLastError());
  }
  return layer_grads<RowPaired>(p, b, X, p.xs ? X8->codes : nullptr, b.dy, s, T, have_t, dX, dL1, dL2, grad_bf16, stream);
}

hipError_t linear_backward_int8(const NF4View& W, const NF4Table& tab, const Int8Values& X8, const uint16_t* dY, int64_t M,
                                const uint16_t* L1, const uint16_t* L2, int r, float s, const uint16_t* T, uint16_t* dX,
                                void* dL1, void* dL2, bool grad_bf16, void* ws, hipStream_t stream) {
  const int64_t K = W.cols, N = W.rows;
  if (M == 0) return zero_grads(K * r, r * N, dL1, dL2, grad_bf16, stream);
  const LayerBuffers b(linear_int8_workspace_layout(M, K, N, r), ws);
  LayerPrep p{};
  p.n = 1;
  p.M = M;
  p.K = K;
  p.N = N;
  p.Np = gd_cdiv(N, 64) * 64;
  p.r = r;
  p.rp = (int)gd_cdiv(r, 64) * 64;
  p.W[0] = W;
  p.tab[0] = tab;
  p.wd = dX ? b.wd : nullptr;
  p.L1 = L1;
  p.L2 = L2;
  p.l1t = b.l1t;
  p.l2p = b.l2p;
  lay_int8(p, b, X8, !T);
  if (p.Np != N) {
    p.dy = dY;
    p.dyp = b.dy;
    dY = b.dy;
  }
  GD_TRY(launch_layer_prep(p, stream));
  return layer_grads<RowDown>(p, b, b.x, p.xs ? X8.codes : nullptr, dY, s, T, T != nullptr, dX, dL1, dL2, grad_bf16, stream);
}

}  // namespace qlora
