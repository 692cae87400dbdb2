// Forward of the linear with an adapter per row for M <= 128 rows (decode
// steps and short prefills), for gfx950:
//
//   Y[m] = X[m] Wd^T + bf16(s_a X[m] L1_a) L2_a,   a = ids[m]
//
// Three launches, none of which needs the rows grouped beforehand: a
// workgroup stands for one row m and takes that row's group, if the row is
// the first, 17th, 33rd ... of the rows with its id (SmallGroup); the others
// end at once.
//
//   small_multi_t_kernel       T partials over K-slices of 512 (fp32)
//   the 4-bit weight           midm.hip's pass over the base weight (K-slice
//                              partials), or for few rows the GEMV, which
//                              also adds the adapters (gemv.hip)
//   small_multi_finish_kernel  Y = bf16(the partials' sum + s_a T L2_a), for
//                              up to 16 rows of one adapter and 512 columns:
//                              an adapter's L2 is read once per 16 rows
// At these sizes the weight stream (0.52 B per weight) and the live adapters
// are all there is to read; the launches' latency is the rest.
#include "common.h"
#include "launch.h"

namespace qlora {

namespace {

constexpr int kGroup = 16;        // rows per workgroup = MFMA rows

// The rows of one adapter that workgroup `m` takes: rows[0 .. n). n = 0: not a
// group's first row. Threads of the whole workgroup; M <= 128.
struct SmallGroup {
  int a, n;
  bool has;                       // the rows have an adapter
};

template <int THREADS>
__device__ __forceinline__ SmallGroup small_group(const int32_t* __restrict__ ids, int M, int A, int m, int* rows) {
  static_assert(THREADS >= 128, "one id per thread");
  __shared__ int s_before[4];     // of waves 0 and 1: rows of the group below m, and in all before the wave
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int own = ids[m];
  const bool own_has = own >= 0 && own < A;
  bool same = false;
  if (tid < M && tid < 128) {
    const int v = ids[tid];
    same = (v >= 0 && v < A) ? v == own : !own_has;   // rows without an adapter are one group
  }
  const unsigned long long b = __ballot(same);
  if (wave < 2 && lane == 0) {
    const int at = m - 64 * wave;                     // rows of this wave below m
    s_before[wave] = __popcll(at <= 0 ? 0ull : at >= 64 ? b : b & ((1ull << at) - 1ull));
    s_before[2 + wave] = __popcll(b);
  }
  __syncthreads();
  const int rank = s_before[0] + s_before[1];         // rows of the group before m
  const int all = s_before[2] + s_before[3];
  SmallGroup g{own, 0, own_has};
  if (rank % kGroup != 0) return g;                   // uniform
  g.n = all - rank < kGroup ? all - rank : kGroup;
  if (same) {
    const int pos = (wave == 1 ? s_before[2] : 0) + __popcll(b & ((1ull << lane) - 1ull)) - rank;
    if (pos >= 0 && pos < kGroup) rows[pos] = tid;
  }
  __syncthreads();
  return g;
}

// T partials: part[slice][m][j] over k-slices of 512; the layout and the
// arithmetic of the single adapter's small_t_partial_kernel. Rows without an
// adapter are not written.
constexpr int kTWaves = 16, kTRows = 32, kTK = kTWaves * kTRows;

__global__ __launch_bounds__(64 * kTWaves) void small_multi_t_kernel(const uint16_t* __restrict__ X, int M, int K,
                                                                     const int32_t* __restrict__ ids, int A,
                                                                     const uint16_t* __restrict__ L1, int r,
                                                                     float* __restrict__ part) {
  __shared__ float red[kTWaves][16][64];
  __shared__ int rows[kGroup];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const SmallGroup g = small_group<64 * kTWaves>(ids, M, A, (int)blockIdx.z, rows);
  if (g.n == 0 || !g.has) return;                     // uniform
  const uint16_t* B = L1 + (int64_t)g.a * K * r;
  const int kw = (int)blockIdx.x * kTK + wave * kTRows + 8 * (lane >> 4);
  const int row = lane & 15;
  const int j0 = (int)blockIdx.y * 64;
  u32x4_t xa = {0u, 0u, 0u, 0u};
  if (row < g.n && kw < K) xa = *reinterpret_cast<const u32x4_t*>(X + (int64_t)rows[row] * K + kw);  // K % 64 == 0
  uint32_t h[4][8];  // all loads first (one round trip)
#pragma unroll
  for (int jt = 0; jt < 4; ++jt) {
    const int j = j0 + 16 * jt + row;
    const bool in = j < r && kw < K;
    const uint16_t* lp = B + (in ? (int64_t)kw * r + j : 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[jt][i] = lp[in ? (int64_t)i * r : 0];
    if (!in) {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[jt][i] = 0u;
    }
  }
#pragma unroll
  for (int jt = 0; jt < 4; ++jt) {
    const u32x4_t b = {h[jt][0] | (h[jt][1] << 16), h[jt][2] | (h[jt][3] << 16), h[jt][4] | (h[jt][5] << 16),
                       h[jt][6] | (h[jt][7] << 16)};
    const f32x4_t acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, xa),
                                                                __builtin_bit_cast(bf16x8_t, b),
                                                                f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
    // register i of lane l: row 4 (l/16) + i, column j0 + 16 jt + l%16
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][4 * (lane >> 4) + i][16 * jt + row] = acc[i];
  }
  __syncthreads();
  if (wave < g.n && j0 + lane < r) {  // thread (row, lane) sums the waves in order
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kTWaves; ++w) v += red[w][wave][lane];
    part[((int64_t)blockIdx.x * M + rows[wave]) * r + j0 + lane] = v;
  }
}

// Y = bf16(sum_z base[z][m][n] + sum_j bf16(s_a T[m][j]) L2_a[j][n]): 512
// columns, 8 per lane, up to 16 rows of one group, 4 per wave. The slices of T
// and of the base are added in order; workgroup column 0 writes T_out.
constexpr int kFinCols = 512;
constexpr int kFinRank = 256;

__global__ __launch_bounds__(256) void small_multi_finish_kernel(const float* __restrict__ base, int S, int M, int N,
                                                                 const int32_t* __restrict__ ids, int A,
                                                                 const float* __restrict__ tpart, int Z, int r,
                                                                 const uint16_t* __restrict__ L2,
                                                                 const float* __restrict__ scale,
                                                                 uint16_t* __restrict__ Y,
                                                                 uint16_t* __restrict__ T_out) {
  __shared__ int rows[kGroup];
  __shared__ float sT[kGroup][kFinRank];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const SmallGroup g = small_group<256>(ids, M, A, (int)blockIdx.y, rows);
  if (g.n == 0) return;                               // uniform
  const int n = (int)blockIdx.x * kFinCols + 8 * lane;
  const bool in = n < N;                              // N % 8 == 0
  const int nc = in ? n : 0;
  float acc[4][8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int i = wave * 4 + q;
    const int64_t row = rows[i < g.n ? i : 0];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[q][e] = 0.0f;
    for (int z = 0; z < S; ++z) {
      const float* p = base + ((int64_t)z * M + row) * N + nc;
      const f32x4_t a = *reinterpret_cast<const f32x4_t*>(p), b = *reinterpret_cast<const f32x4_t*>(p + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[q][e] += a[e];
        acc[q][4 + e] += b[e];
      }
    }
  }
  if (g.has) {
    const float s = scale[g.a];
    for (int i = tid; i < g.n * r; i += 256) {
      const int k = i / r, j = i - k * r;
      float v = 0.0f;
      for (int z = 0; z < Z; ++z) v += tpart[((int64_t)z * M + rows[k]) * r + j];
      sT[k][j] = bf16_to_f32(f32_to_bf16(s * v));
      if (T_out && blockIdx.x == 0) T_out[(int64_t)rows[k] * r + j] = f32_to_bf16(v);
    }
  } else if (T_out && blockIdx.x == 0) {
    for (int i = tid; i < g.n * r; i += 256) T_out[(int64_t)rows[i / r] * r + i % r] = 0;
  }
  __syncthreads();
  if (g.has) {
    const uint16_t* B = L2 + (int64_t)g.a * r * N + nc;
#pragma unroll 8
    for (int j = 0; j < r; ++j) {
      const u32x4_t w = *reinterpret_cast<const u32x4_t*>(B + (int64_t)j * N);
      const uint32_t v[4] = {w.x, w.y, w.z, w.w};
      float l[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        l[2 * e] = __uint_as_float(v[e] << 16);
        l[2 * e + 1] = __uint_as_float(v[e] & 0xFFFF0000u);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float t = sT[wave * 4 + q][j];          // rows past the group: not stored
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[q][e] = __builtin_fmaf(t, l[e], acc[q][e]);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int i = wave * 4 + q;
    if (i < g.n && in)
      *reinterpret_cast<u32x4_t*>(Y + (int64_t)rows[i] * N + n) =
          u32x4_t{pack_bf16x2(acc[q][0], acc[q][1]), pack_bf16x2(acc[q][2], acc[q][3]),
                  pack_bf16x2(acc[q][4], acc[q][5]), pack_bf16x2(acc[q][6], acc[q][7])};
  }
}

}  // namespace

int64_t multi_small_t_floats(int64_t M, int64_t K, int r) { return (K + kTK - 1) / kTK * M * r; }
int multi_small_t_slices(int64_t K) { return (int)((K + kTK - 1) / kTK); }

hipError_t launch_multi_small_t(const uint16_t* X, int64_t M, int64_t K, const MultiIds& mi, const uint16_t* L1, int r,
                                float* part, hipStream_t stream) {
  hipLaunchKernelGGL(small_multi_t_kernel,
                     dim3((unsigned)multi_small_t_slices(K), (unsigned)((r + 63) / 64), (unsigned)M),
                     dim3(64 * kTWaves), 0, stream, X, (int)M, (int)K, mi.ids, mi.A, L1, r, part);
  return hipGetLastError();
}

hipError_t launch_multi_small_finish(const float* base, int S, int64_t M, int64_t N, const MultiIds& mi,
                                     const float* tpart, int Z, int r, const uint16_t* L2, uint16_t* Y,
                                     uint16_t* T_out, hipStream_t stream) {
  hipLaunchKernelGGL(small_multi_finish_kernel, dim3((unsigned)((N + kFinCols - 1) / kFinCols), (unsigned)M), dim3(256),
                     0, stream, base, S, (int)M, (int)N, mi.ids, mi.A, tpart, Z, r, L2, mi.scale, Y, T_out);
  return hipGetLastError();
}

}  // namespace qlora
