// The QLoRA linear with an adapter per row, for gfx950:
//
//   Y[m]  = X[m] Wd^T + s_a (X[m] L1_a) L2_a,               a = row_adapter[m]
//   dX[m] = dY[m] Wd  + s_a (dY[m] L2_a^T) L1_a^T
//   dL1_a = s_a sum_{m of a} X[m]^T (dY[m] L2_a^T),  dL2_a = s_a sum_{m of a} (X[m] L1_a)^T dY[m]
//
// Rows whose id lies outside [0, A) use the base alone. This file holds the
// path for M > 128 rows and the backward pass; gemv1.hip, gemv.hip and
// multi_small.hip hold the small ones.
//
//   route_kernel      groups the rows by adapter (see multi.h)
//   multi_nt_kernel   T = X L1_a or U = dY L2_a^T over 128-row pieces of the
//                     grouped rows, split over the reduction into fp32 partials
//   multi_tr_kernel   sums them, scales each row by its s_a, rounds to bf16
//   the dense GEMM    (dense_gemm.hip) walks the grouped rows; its adapter
//                     stages run over the segments that meet the tile
//   multi_tn_kernel   dL1_a, dL2_a: per piece of a segment, the product with
//                     the reduction down the rows
// Rows are gathered where a kernel loads them (a row's 128-byte stage slices
// are whole cache lines, so the gather costs no bandwidth), and every row
// buffer stays in the caller's order. All sums run in a fixed order.
#include "common.h"
#include "launch.h"
#include "multi.h"

namespace qlora {

namespace {

typedef __attribute__((address_space(3))) void lds_void_t;

__device__ __attribute__((aligned(16))) uint32_t g_multi_zero[4];  // zero-initialised copy source

// ---- route ---------------------------------------------------------------------

constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / 64;

__device__ __forceinline__ int block_sum(int v, int* s) {   // 1024 threads; s: kRouteWaves ints
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  int t = 0;
#pragma unroll
  for (int w = 0; w < kRouteWaves; ++w) t += s[w];
  return t;
}

// Workgroup a < A: adapter a; workgroup A: the rows without one. Each reads
// all ids (from the L2 after the first): it counts the rows and the distinct
// adapters below its own, which are its place and its segment number, then
// writes its rows in order. slot (optional) receives an adapter's segment.
__global__ __launch_bounds__(kRouteThreads) void route_kernel(const int32_t* __restrict__ ids, int M, int A,
                                                              int32_t* __restrict__ perm, int32_t* __restrict__ start,
                                                              int32_t* __restrict__ adapter,
                                                              int32_t* __restrict__ count,
                                                              int32_t* __restrict__ slot) {
  extern __shared__ uint32_t seen[];                // A bits
  __shared__ int s_sum[kRouteWaves], s_wave[kRouteWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int a = (int)blockIdx.x;
  const int words = (A + 31) / 32;
  for (int i = tid; i < words; i += kRouteThreads) seen[i] = 0u;
  __syncthreads();
  int below = 0, mine = 0;
  for (int i = tid; i < M; i += kRouteThreads) {
    const int v = ids[i];
    const bool has = v >= 0 && v < A;
    if (has && v < a) {
      ++below;
      atomicOr(&seen[v >> 5], 1u << (v & 31));      // the same bits in any order
    }
    mine += a < A ? v == a : !has;
  }
  below = block_sum(below, s_sum);
  mine = block_sum(mine, s_sum);                    // its barriers also publish `seen`
  int rank = 0;
  for (int i = tid; i < words; i += kRouteThreads) rank += __popc(seen[i]);
  rank = block_sum(rank, s_sum);
  if (tid == 0) {
    if (a == A) {
      count[0] = rank;
      start[rank] = below;
    } else if (mine > 0) {
      adapter[rank] = a;
      start[rank] = below;
      if (slot) slot[a] = rank;
    }
  }
  if (mine == 0) return;                            // uniform
  int at = below;
  for (int i0 = 0; i0 < M; i0 += kRouteThreads) {
    const int i = i0 + tid;
    const int v = i < M ? ids[i] : 0;
    const bool take = i < M && (a < A ? v == a : !(v >= 0 && v < A));
    const unsigned long long b = __ballot(take);
    __syncthreads();
    if (lane == 0) s_wave[wave] = __popcll(b);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kRouteWaves; ++w) {
      const int c = s_wave[w];
      before += w < wave ? c : 0;
      all += c;
    }
    if (take) perm[at + before + __popcll(b & ((1ull << lane) - 1ull))] = i;
    at += all;
  }
}

// ---- adapter operands of the dense GEMM ---------------------------------------------

// out[k] = the transpose of L2 of segment k: [N][rp], columns >= r zero. One
// workgroup per 64 columns n and 64 ranks of one segment.
__global__ __launch_bounds__(256) void multi_l2t_kernel(const uint16_t* __restrict__ L2, int64_t N, int r, int rp,
                                                        RouteView rv, uint16_t* __restrict__ out) {
  __shared__ uint16_t tile[64][64 + 2];
  const int k = blockIdx.z;
  if (k >= rv.count[0]) return;                     // uniform
  const uint16_t* src = L2 + (int64_t)rv.adapter[k] * r * N;
  const int64_t n0 = (int64_t)blockIdx.x * 64;
  const int j0 = blockIdx.y * 64;
  const int t = threadIdx.x;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int j = (t >> 3) + 32 * u, c = (t & 7) * 8;
    u32x4_t v = {0u, 0u, 0u, 0u};
    if (j0 + j < r && n0 + c < N) v = *reinterpret_cast<const u32x4_t*>(src + (int64_t)(j0 + j) * N + n0 + c);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) tile[c + e][j] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int n = (t >> 3) + 32 * u, c = (t & 7) * 8;
    if (n0 + n >= N) continue;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = (uint32_t)tile[n][c + 2 * e] | ((uint32_t)tile[n][c + 2 * e + 1] << 16);
    *reinterpret_cast<u32x4_t*>(out + ((int64_t)k * N + n0 + n) * rp + j0 + c) = u32x4_t{w[0], w[1], w[2], w[3]};
  }
}

// out[k] = L1 of segment k with its columns padded to rp: [K][rp].
__global__ __launch_bounds__(256) void multi_l1p_kernel(const uint16_t* __restrict__ L1, int64_t K, int r, int rp,
                                                        RouteView rv, uint16_t* __restrict__ out) {
  const int k = blockIdx.y;
  if (k >= rv.count[0]) return;
  const uint16_t* src = L1 + (int64_t)rv.adapter[k] * K * r;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;   // 16-byte piece of the output
  const int per = rp / 8;
  if (i >= K * per) return;
  const int64_t row = i / per;
  const int c = (int)(i - row * per) * 8;
  u32x4_t v = {0u, 0u, 0u, 0u};
  if (c < r) v = *reinterpret_cast<const u32x4_t*>(src + row * r + c);
  *reinterpret_cast<u32x4_t*>(out + ((int64_t)k * K + row) * rp + c) = v;
}

// ---- pieces shared by the two adapter products -----------------------------------------

constexpr int SK = 64;       // reduction per stage
constexpr int SJ = 64;       // ranks per tile
constexpr int SM = 128;      // rows (nt) or columns (tn) per tile
constexpr int kThreads = 256;
constexpr int kStages = 3;

// 16-byte chunk c of a 128-byte LDS row sits at c ^ swz(row): 16 consecutive
// rows' fragment reads fall on distinct bank groups.
__device__ __forceinline__ int row_swz(int row) { return ((row >> 1) ^ (row >> 4)) & 7; }
__device__ __forceinline__ int row_off(int row, int chunk) { return row * SK + ((chunk ^ row_swz(row)) << 3); }
// The same for operands read through the transpose read: the four rows that
// one read of 32 lanes touches fall on distinct bank groups (256-byte rows),
// or rows m and m + 2 apart (128-byte rows).
__device__ __forceinline__ int tr_swz256(int m) { return (m & 3) << 2; }
__device__ __forceinline__ int tr_swz128(int m) { return ((m >> 1) & 1) << 2; }

// One 16-byte copy per lane into 1 KB of LDS. Issued from inline assembly: the
// caller's vmcnt before each stage's barrier is the only wait on the copies.
__device__ __forceinline__ void copy16(const void* src, const void* lds) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void_t*)lds);
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" :: "v"(src), "s"(m0) : "memory", "m0");
}

typedef short v4i16_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ v4i16_t read_tr(const char* lds) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16_t*)(lds_void_t*)lds);
}
__device__ __forceinline__ bf16x8_t frag_tr(const char* r0, const char* r4) {   // rows m .. m+3 and m+4 .. m+7
  return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(read_tr(r0), read_tr(r4), 0, 1, 2, 3, 4, 5, 6, 7));
}

struct NtArgs {
  const uint16_t* A;      // [M][lda], the streamed rows
  const uint16_t* B;      // per adapter: [r][ldb] (BT = false) or [len][r] (BT = true)
  float* C;               // [Z][M][rp]; columns < r written, rows of segments only
  int64_t lda, ldb, b_stride;
  int64_t M, len, split;  // reduction length, and per slice
  int r, rp;
  RouteView rv;
};

// C[z][m][j] = sum over slice z of A[m][i] B_a[j][i]: 128 grouped rows of one
// segment by 64 ranks; 4 waves of 32 rows; the copies of two stages are in
// flight while a third is multiplied. With BT the adapter's operand has its
// ranks contiguous (L1 as stored) and its fragments come through the LDS
// transpose read; without, its reduction is contiguous (L2 as stored).
template <bool BT>
__global__ __launch_bounds__(kThreads) void multi_nt_kernel(NtArgs p) {
  __shared__ __attribute__((aligned(1024))) uint16_t sA[kStages][SM * SK];
  __shared__ __attribute__((aligned(1024))) uint16_t sB[kStages][SJ * SK];
  __shared__ int s_row[SM];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const RoutePiece pc = route_piece(p.rv, (int)blockIdx.x, SM);
  if (pc.hi <= pc.lo) return;                       // uniform: no barrier was reached
  const int j0 = (int)blockIdx.y * SJ;
  const int64_t z0 = (int64_t)blockIdx.z * p.split;
  const int64_t z1 = z0 + p.split < p.len ? z0 + p.split : p.len;
  const int ns = z0 < z1 ? (int)((z1 - z0 + SK - 1) / SK) : 0;
  if (tid < SM) s_row[tid] = p.rv.perm[pc.lo + tid < pc.hi ? pc.lo + tid : pc.hi - 1];
  __syncthreads();
  const char* zero = reinterpret_cast<const char*>(g_multi_zero);
  const uint16_t* B = p.B + (int64_t)p.rv.adapter[pc.k] * p.b_stride;
  const int lr = lane >> 3;

  const uint16_t* a_src[4];
  int a_col[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int rl = (wave * 4 + q) * 8 + lr;
    a_col[q] = ((lane & 7) ^ row_swz(rl)) * 8;
    a_src[q] = p.A + (int64_t)s_row[rl] * p.lda + z0 + a_col[q];
  }
  const uint16_t* b_src[2];
  int b_col[2];
  bool b_in[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int rl = (wave * 2 + q) * 8 + lr;
    if constexpr (BT) {
      const int j = j0 + 8 * ((lane & 7) ^ tr_swz128(rl));
      b_in[q] = j < p.r;
      b_col[q] = rl;                                // the row's place along the reduction
      b_src[q] = B + (z0 + rl) * p.r + (b_in[q] ? j : 0);
    } else {
      b_col[q] = ((lane & 7) ^ row_swz(rl)) * 8;
      b_in[q] = j0 + rl < p.r;
      b_src[q] = B + (int64_t)(b_in[q] ? j0 + rl : 0) * p.ldb + z0 + b_col[q];
    }
  }
  auto issue = [&](int st) {
    const int64_t left = z1 - z0 - (int64_t)st * SK;   // reduction left from this stage on
    const int buf = st % kStages;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      copy16(a_col[q] < left ? reinterpret_cast<const char*>(a_src[q] + (int64_t)st * SK) : zero,
             sA[buf] + (wave * 4 + q) * 8 * SK);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int64_t step = (int64_t)st * SK * (BT ? p.r : 1);
      copy16(b_in[q] && b_col[q] < left ? reinterpret_cast<const char*>(b_src[q] + step) : zero,
             sB[buf] + (wave * 2 + q) * 8 * SK);
    }
  };

  f32x16_t acc[2];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[t][v] = 0.0f;
  // transpose-read places (as in multi_tn_kernel)
  const int jl = lane & 15, rb = 8 * (lane >> 5) + (jl >> 2), cb = 16 * ((lane >> 4) & 1) + 4 * (jl & 3);
  auto b_tr = [&](const char* base, int row, int t) {
    const int c = 32 * t + cb;
    return base + row * (SJ * 2) + (((c >> 3) ^ tr_swz128(row)) << 4) + ((c & 7) << 1);
  };

#pragma unroll
  for (int s = 0; s < kStages - 1; ++s)
    if (s < ns) issue(s);
  for (int st = 0; st < ns; ++st) {
    const int buf = st % kStages;
    if (st + 1 < ns) asm volatile("s_waitcnt vmcnt(6)" ::: "memory");  // the next stage's 6 copies may stay in flight
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (st + kStages - 1 < ns) issue(st + kStages - 1);
    const char* bb = reinterpret_cast<const char*>(sB[buf]);
#pragma unroll
    for (int kk = 0; kk < SK / 16; ++kk) {
      const int ch = 2 * kk + (lane >> 5);
      const bf16x8_t a = *reinterpret_cast<const bf16x8_t*>(sA[buf] + row_off(wave * 32 + (lane & 31), ch));
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        bf16x8_t b;
        if constexpr (BT) b = frag_tr(b_tr(bb, 16 * kk + rb, t), b_tr(bb, 16 * kk + rb + 4, t));
        else b = *reinterpret_cast<const bf16x8_t*>(sB[buf] + row_off(t * 32 + (lane & 31), ch));
        acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc[t], 0, 0, 0);
      }
    }
  }
  // lane l, register v -> row (v%4) + 4(l/32) + 8(v/4), column l%32
  float* C = p.C + (int64_t)blockIdx.z * p.M * p.rp;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int j = j0 + t * 32 + (lane & 31);
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int rl = wave * 32 + (v & 3) + 4 * (lane >> 5) + 8 * (v >> 2);
      if (pc.lo + rl < pc.hi && j < p.r) C[(int64_t)s_row[rl] * p.rp + j] = acc[t][v];
    }
  }
}

// From the partials P [Z][M][rp]: scaled [M][rp] = bf16(s_a sum) and plain
// [M][r] = bf16(sum), either may be null; rows without an adapter and columns
// >= r are zero. 4 columns per thread.
__global__ __launch_bounds__(256) void multi_tr_kernel(const float* __restrict__ P, int Z, int64_t M, int r, int rp,
                                                       const int32_t* __restrict__ ids, int A,
                                                       const float* __restrict__ scale, uint16_t* __restrict__ scaled,
                                                       uint16_t* __restrict__ plain) {
  const int w4 = rp / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= M * w4) return;
  const int64_t m = i / w4;
  const int j = (int)(i - m * w4) * 4;
  const int a = ids[m];
  f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
  float s = 0.0f;
  if (a >= 0 && a < A && j < r) {
    s = scale[a];
    const float* p = P + m * rp + j;
    int z = 0;
    for (; z + 4 <= Z; z += 4) {  // loads of 4 slices in flight, added in order
      f32x4_t q[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) q[u] = *reinterpret_cast<const f32x4_t*>(p + (int64_t)(z + u) * M * rp);
#pragma unroll
      for (int u = 0; u < 4; ++u) v += q[u];
    }
    for (; z < Z; ++z) v += *reinterpret_cast<const f32x4_t*>(p + (int64_t)z * M * rp);
  }
  if (plain && j < r)
    *reinterpret_cast<u32x2_t*>(plain + m * r + j) = u32x2_t{pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
  if (scaled)
    *reinterpret_cast<u32x2_t*>(scaled + m * rp + j) = u32x2_t{pack_bf16x2(s * v.x, s * v.y), pack_bf16x2(s * v.z, s * v.w)};
}

struct TnArgs {
  const uint16_t* L;      // [M][ldl]: X or dY
  const uint16_t* S;      // [M][lds]: U or T, r columns used
  void* out;              // per adapter: [W][r] (RANKS_IN = true) or [r][W]
  float* part;            // per piece and rank tile: [W][64] or [64][W]
  const float* scale;     // factor per adapter, or null
  int64_t ldl, lds, W, slab;   // slab: floats per piece (all its rank tiles)
  int r, rows;            // rows per piece
  bool out_bf16;
  RouteView rv;
};

constexpr int kTnLRow = SM * 2, kTnSRow = SJ * 2;
constexpr int kTnLBytes = SK * kTnLRow;
constexpr int kTnStageBytes = kTnLBytes + SK * kTnSRow;
constexpr int kTnRows = 2048;   // most rows of a piece: their list takes 8 KB, and two workgroups still fit in a CU's LDS

// One value of the gradients' layout: RANKS_IN: [w][j] with row length `in`.
template <bool RANKS_IN>
__device__ __forceinline__ int64_t tn_at(int64_t w, int j, int64_t W, int in) {
  return RANKS_IN ? w * in + j : (int64_t)j * W + w;
}

// sum over the rows m of one piece of a segment of L[m][w] S[m][j], for 128
// columns w and 64 ranks j. Both operands are copied to LDS as they lie (rows
// along m) and read through the transpose read. A segment of one piece is
// finished here; the pieces of a longer one go to `part`. RANKS_IN puts the
// ranks on the lanes (a row of dL1 is r contiguous values), otherwise the
// columns (a row of dL2 is W contiguous values): the same products with the
// MFMA operands exchanged.
template <bool RANKS_IN>
__global__ __launch_bounds__(kThreads) void multi_tn_kernel(TnArgs p) {
  __shared__ __attribute__((aligned(1024))) char ring[kStages * kTnStageBytes];
  __shared__ int s_row[kTnRows];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const RoutePiece pc = route_piece(p.rv, (int)blockIdx.z, p.rows);
  if (pc.hi <= pc.lo) return;                       // uniform: no barrier was reached
  const int64_t c0 = (int64_t)blockIdx.x * SM;
  const int j0 = (int)blockIdx.y * SJ;
  const int ns = (pc.hi - pc.lo + SK - 1) / SK;
  const char* zero = reinterpret_cast<const char*>(g_multi_zero);

  // L: instruction i of wave w moves rows 4 (4w + i) .. +3, lane -> row + lane / 16, chunk lane % 16;
  // S: rows 8 (2w + i) .. +7, lane -> row + lane / 8, chunk lane % 8
  int64_t l_col[4], s_col[2];
  bool s_in[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 4 * (4 * wave + i) + (lane >> 4);
    int64_t c = c0 + 8 * ((lane & 15) ^ tr_swz256(row));
    if (c > p.W - 8) c = p.W - 8;                   // W % 8 == 0; columns past W are not stored
    l_col[i] = c;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = 8 * (2 * wave + i) + (lane >> 3);
    const int j = j0 + 8 * ((lane & 7) ^ tr_swz128(row));
    s_in[i] = j < p.r;
    s_col[i] = s_in[i] ? j : 0;
  }
  for (int i = tid; i < pc.hi - pc.lo; i += kThreads) s_row[i] = p.rv.perm[pc.lo + i];
  __syncthreads();
  const int n = pc.hi - pc.lo;
  auto issue = [&](int st) {
    char* buf = ring + (st % kStages) * kTnStageBytes;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = st * SK + 4 * (4 * wave + i) + (lane >> 4);
      copy16(m < n ? reinterpret_cast<const char*>(p.L + (int64_t)s_row[m < n ? m : 0] * p.ldl + l_col[i]) : zero,
             buf + (4 * wave + i) * 1024);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = st * SK + 8 * (2 * wave + i) + (lane >> 3);
      copy16(m < n && s_in[i] ? reinterpret_cast<const char*>(p.S + (int64_t)s_row[m < n ? m : 0] * p.lds + s_col[i]) : zero,
             buf + kTnLBytes + (2 * wave + i) * 1024);
    }
  };

  f32x16_t acc[2];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[t][v] = 0.0f;
  // transpose read: lane j of a 16-lane group addresses row m0 + j / 4, columns cb + 4 (j % 4) .. +3 and
  // receives rows m0 .. m0 + 3 of column cb + j
  const int jl = lane & 15, rb = 8 * (lane >> 5) + (jl >> 2);
  const int cl = wave * 32 + 16 * ((lane >> 4) & 1) + 4 * (jl & 3), cs = 16 * ((lane >> 4) & 1) + 4 * (jl & 3);
  auto l_at = [&](const char* b, int row) {
    return b + row * kTnLRow + (((cl >> 3) ^ tr_swz256(row)) << 4) + ((cl & 7) << 1);
  };
  auto s_at = [&](const char* b, int row, int t) {
    const int c = 32 * t + cs;
    return b + kTnLBytes + row * kTnSRow + (((c >> 3) ^ tr_swz128(row)) << 4) + ((c & 7) << 1);
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s)
    if (s < ns) issue(s);
  for (int st = 0; st < ns; ++st) {
    if (st + 1 < ns) asm volatile("s_waitcnt vmcnt(6)" ::: "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (st + kStages - 1 < ns) issue(st + kStages - 1);
    const char* buf = ring + (st % kStages) * kTnStageBytes;
#pragma unroll
    for (int kk = 0; kk < SK / 16; ++kk) {
      const int r0 = 16 * kk + rb;
      const bf16x8_t l = frag_tr(l_at(buf, r0), l_at(buf, r0 + 4));
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const bf16x8_t s = frag_tr(s_at(buf, r0, t), s_at(buf, r0 + 4, t));
        acc[t] = RANKS_IN ? __builtin_amdgcn_mfma_f32_32x32x16_bf16(l, s, acc[t], 0, 0, 0)
                          : __builtin_amdgcn_mfma_f32_32x32x16_bf16(s, l, acc[t], 0, 0, 0);
      }
    }
  }
  const int s0 = p.rv.start[pc.k], s1 = p.rv.start[pc.k + 1];
  const bool whole = s1 - s0 <= p.rows;
  const int a = p.rv.adapter[pc.k];
  const float f = whole && p.scale ? p.scale[a] : 1.0f;
  float* part = p.part + (int64_t)blockIdx.z * p.slab + (int64_t)j0 * p.W;
  const int64_t out0 = (int64_t)a * p.W * p.r;
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int row = (v & 3) + 4 * (lane >> 5) + 8 * (v >> 2), col = lane & 31;
      const int64_t w = c0 + wave * 32 + (RANKS_IN ? row : col);
      const int j = 32 * t + (RANKS_IN ? col : row);
      if (w >= p.W || j0 + j >= p.r) continue;
      const float x = acc[t][v];
      if (!whole) {
        part[tn_at<RANKS_IN>(w, j, p.W, SJ)] = x;
      } else {
        const int64_t o = out0 + tn_at<RANKS_IN>(w, j0 + j, p.W, p.r);
        if (p.out_bf16) static_cast<uint16_t*>(p.out)[o] = f32_to_bf16(f * x);
        else static_cast<float*>(p.out)[o] = f * x;
      }
    }
}

// The gradients that multi_tn_kernel left open: the sums of a segment's
// several pieces, in order, and zeros for adapters without rows. Workgroup
// (x, a); 4 consecutive output values per thread and step.
template <bool RANKS_IN>
__global__ __launch_bounds__(256) void multi_tn_reduce_kernel(TnArgs p) {
  const int a = (int)blockIdx.y, lane = threadIdx.x & 63;
  const int n = p.rv.count[0];
  int k = -1;
  for (int base = 0; base < n; base += 64) {
    const int i = base + lane;
    const unsigned long long hit = __ballot(i < n && p.rv.adapter[i < n ? i : 0] == a);
    if (hit) k = base + __builtin_ctzll(hit);
  }
  k = __builtin_amdgcn_readfirstlane(k);
  int first = 0, pieces = 0;
  if (k >= 0) {
    const int s0 = p.rv.start[k], s1 = p.rv.start[k + 1];
    pieces = (s1 - s0 + p.rows - 1) / p.rows;
    first = s0 / p.rows + k;
    if (pieces == 1) return;
  }
  const float f = p.scale ? p.scale[a] : 1.0f;
  const int64_t total = p.W * p.r;                  // r % 8 == 0, W % 8 == 0: 4 values never leave a row
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < total; i += (int64_t)gridDim.x * 1024) {
    f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (pieces > 0) {
      const int64_t w = RANKS_IN ? i / p.r : i % p.W;
      const int j = (int)(RANKS_IN ? i % p.r : i / p.W);
      const float* src = p.part + (int64_t)first * p.slab + (int64_t)(j / SJ) * SJ * p.W + tn_at<RANKS_IN>(w, j % SJ, p.W, SJ);
      for (int q = 0; q < pieces; ++q) v += *reinterpret_cast<const f32x4_t*>(src + q * p.slab);
    }
    const int64_t o = (int64_t)a * total + i;
    if (p.out_bf16)
      *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(p.out) + o) =
          u32x2_t{pack_bf16x2(f * v.x, f * v.y), pack_bf16x2(f * v.z, f * v.w)};
    else
      *reinterpret_cast<f32x4_t*>(static_cast<float*>(p.out) + o) = f32x4_t{f * v.x, f * v.y, f * v.z, f * v.w};
  }
}

__global__ __launch_bounds__(256) void multi_zero_kernel(uint32_t* __restrict__ p, int64_t words) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words; i += (int64_t)gridDim.x * 256) p[i] = 0u;
}

// dst [M][ldd] = src [M][cols] with columns cols .. ldd zero (both multiples of 8).
__global__ __launch_bounds__(256) void multi_pad_rows_kernel(const uint16_t* __restrict__ src, int64_t M, int64_t cols,
                                                             uint16_t* __restrict__ dst, int64_t ldd) {
  const int64_t per = ldd / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < M * per; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / per, c = (i - m * per) * 8;
    u32x4_t v = {0u, 0u, 0u, 0u};
    if (c < cols) v = *reinterpret_cast<const u32x4_t*>(src + m * cols + c);
    *reinterpret_cast<u32x4_t*>(dst + m * ldd + c) = v;
  }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
unsigned capped(int64_t blocks) { return (unsigned)(blocks < 1 ? 1 : blocks > 16384 ? 16384 : blocks); }

// Reduction slices of the NT products: about two workgroups per CU, the
// number that is resident at once.
struct NtSplit {
  int64_t len;
  int Z;
};
NtSplit nt_split(int64_t M, int64_t len, int A, int rp) {
  int64_t tiles = (cdiv(M, SM) + (A < M ? A : M) / 2) * (rp / SJ);
  if (tiles < 1) tiles = 1;
  const int64_t steps = cdiv(len, SK);
  int64_t z = 2 * (int64_t)device_cu_count() / tiles;
  if (z > 16) z = 16;
  if (z > steps) z = steps;
  if (z < 1) z = 1;
  const int64_t per = cdiv(steps, z);
  return NtSplit{per * SK, (int)cdiv(steps, per)};
}

// Rows per piece of the TN products: whole segments up to 2048 rows, so that
// most gradients are written once; fewer when the launch would not fill the
// device (128 columns per workgroup).
int tn_rows(int64_t M, int64_t W, int r) {
  const int64_t tiles = cdiv(W, SM) * cdiv(r, SJ);
  const int64_t want = cdiv(2 * (int64_t)device_cu_count(), tiles);   // pieces
  int64_t rows = cdiv(cdiv(M, want), SK) * SK;
  if (rows > kTnRows) rows = kTnRows;
  if (rows < 256) rows = 256;
  return (int)rows;
}

int64_t tn_part_floats(int64_t M, int64_t W, int r, int A) {
  const int rows = tn_rows(M, W, r);
  if (M <= rows) return 0;                          // one piece per segment
  return (M / rows + (A < M ? A : M)) * W * cdiv(r, SJ) * SJ;
}

// Per-lane offsets of the GEMM are 32-bit: rows per launch.
int64_t gemm_rows(int64_t M, int64_t widest) {
  const int64_t most = (((int64_t)1 << 31) - 1) / (widest * 2) / 256 * 256;
  return M < most ? M : most;
}

}  // namespace

MultiWorkspace multi_workspace_layout(int64_t M, int64_t K, int64_t N, int r, int A, bool bwd) {
  MultiWorkspace L = {};
  if (!bwd && (M < 1 || multi_small_fits(M, K, N))) {   // the small paths
    L.part_off = 0;
    L.tpart_off = align_up((size_t)multi_small_slices(M, K, N) * M * N * 4, 256);
    const size_t t = (size_t)multi_small_t_floats(M, K, r) * 4, one = gemv1_partial_bytes(K, r);
    L.total = L.tpart_off + align_up((t > one ? t : one) + 1, 256);
    return L;
  }
  const int64_t rp = cdiv(r, 64) * 64, segs = A < M ? A : M, np = cdiv(N, 64) * 64;
  size_t off = 0;
  auto take = [&](int64_t bytes) {
    const size_t at = off;
    off += align_up((size_t)bytes, 256);
    return at;
  };
  L.perm_off = take(M * 4);
  L.start_off = take((segs + 1) * 4);
  L.adapter_off = take(segs * 4);
  L.count_off = take(4);
  L.slot_off = take(A * 4);
  L.perm2_off = take(M * 4);        // the grouping of a part of the rows (more rows than one GEMM launch takes)
  L.start2_off = take((segs + 1) * 4);
  L.adapter2_off = take(segs * 4);
  L.count2_off = take(4);
  L.st_off = take((M + 1) * rp * 2);   // s T or s U, and a row of zeros
  L.t_off = take(bwd ? M * r * 2 : 0);
  const int64_t wide = bwd ? (r % 64 ? segs * K * rp * 2 : 0) : segs * N * rp * 2;
  L.b2_off = take(wide);
  L.wd_off = take(K * np * 2);
  L.dy_off = take(bwd && N % 64 ? M * np * 2 : 0);
  const NtSplit t = nt_split(M, K, A, (int)rp), u = nt_split(M, N, A, (int)rp);
  int64_t part = t.Z * M * rp;
  if (bwd) {
    if (u.Z * M * rp > part) part = u.Z * M * rp;
    const int64_t a = tn_part_floats(M, K, r, A), b = tn_part_floats(M, N, r, A);
    if (a > part) part = a;
    if (b > part) part = b;
  }
  L.part_off = take(part * 4);
  L.total = off;
  return L;
}

namespace {

hipError_t route(const int32_t* ids, int64_t M, int A, char* ws, size_t perm, size_t start, size_t adapter,
                 size_t count, int32_t* slot, RouteView* rv, hipStream_t stream) {
  int32_t* p = reinterpret_cast<int32_t*>(ws + perm);
  int32_t* s = reinterpret_cast<int32_t*>(ws + start);
  int32_t* a = reinterpret_cast<int32_t*>(ws + adapter);
  int32_t* c = reinterpret_cast<int32_t*>(ws + count);
  hipLaunchKernelGGL(route_kernel, dim3((unsigned)(A + 1)), dim3(kRouteThreads), (size_t)(A + 31) / 32 * 4, stream,
                     ids, (int)M, A, p, s, a, c, slot);
  *rv = RouteView{p, s, a, c};
  return hipGetLastError();
}

// scaled [M][rp] and/or plain [M][r] of rows times their adapters' operand.
template <bool BT>
hipError_t rows_by_adapter(const uint16_t* X, int64_t len, const uint16_t* B, int64_t ldb, int64_t b_stride, int64_t M,
                           int r, int rp, int A, const int32_t* ids, const float* scale, const RouteView& rv,
                           float* part, uint16_t* scaled, uint16_t* plain, hipStream_t stream) {
  const NtSplit sp = nt_split(M, len, A, rp);
  NtArgs a;
  a.A = X; a.B = B; a.C = part;
  a.lda = len; a.ldb = ldb; a.b_stride = b_stride;
  a.M = M; a.len = len; a.split = sp.len;
  a.r = r; a.rp = rp; a.rv = rv;
  const int64_t pieces = M / SM + (A < M ? A : M);
  hipLaunchKernelGGL(multi_nt_kernel<BT>, dim3((unsigned)pieces, (unsigned)(rp / SJ), (unsigned)sp.Z), dim3(kThreads),
                     0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(multi_tr_kernel, dim3((unsigned)cdiv(M * rp / 4, 256)), dim3(256), 0, stream, part, sp.Z, M, r, rp,
                     ids, A, scale, scaled, plain);
  return hipGetLastError();
}

// C = X B^T + S_a B2_a^T, in launches of as many rows as 32-bit offsets reach.
// B2's operands lie b2_stride apart, by adapter or (slot) by segment.
hipError_t gemm_by_adapter(const uint16_t* X, int64_t K, const uint16_t* B, int64_t M, int64_t N, const uint16_t* S,
                           const uint16_t* B2, int64_t rp, int64_t b2_stride, const int32_t* slot, uint16_t* C,
                           const int32_t* ids, int A, const RouteView& rv, char* ws, const MultiWorkspace& L,
                           int timing, hipStream_t stream) {
  const int64_t most = gemm_rows(M, K > rp ? K : rp);
  if (most < 1) return hipErrorInvalidValue;
  for (int64_t r0 = 0; r0 < M; r0 += most) {
    const int64_t rows = M - r0 < most ? M - r0 : most;
    MultiSlab slab;
    slab.rv = rv;
    if (rows < M) {
      const hipError_t e = route(ids + r0, rows, A, ws, L.perm2_off, L.start2_off, L.adapter2_off, L.count2_off,
                                 nullptr, &slab.rv, stream);
      if (e != hipSuccess) return e;
    }
    slab.slot = slot;
    slab.zero_row = M - r0;
    slab.b2_stride = b2_stride;
    const hipError_t e = timed(timing, stream, [&] {
      return launch_gemm_nt_multi(X + r0 * K, K, B, K, rows, N, K, S + r0 * rp, B2, rp, slab, C + r0 * N, N, stream);
    });
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t zero_words(void* p, int64_t bytes, hipStream_t stream) {
  hipLaunchKernelGGL(multi_zero_kernel, dim3(capped(cdiv(bytes / 4, 256))), dim3(256), 0, stream,
                     static_cast<uint32_t*>(p), bytes / 4);
  return hipGetLastError();
}

template <bool RANKS_IN>
hipError_t gradient(const uint16_t* L, int64_t W, const uint16_t* S, int64_t lds, int64_t M, int r, int A,
                    const float* scale, const RouteView& rv, float* part, void* out, bool out_bf16,
                    hipStream_t stream) {
  TnArgs a;
  a.L = L; a.S = S; a.out = out; a.part = part; a.scale = scale;
  a.ldl = W; a.lds = lds; a.W = W;
  a.slab = W * cdiv(r, SJ) * SJ;
  a.r = r;
  a.rows = tn_rows(M, W, r);
  a.out_bf16 = out_bf16;
  a.rv = rv;
  const int64_t pieces = M / a.rows + (A < M ? A : M);
  hipLaunchKernelGGL(multi_tn_kernel<RANKS_IN>, dim3((unsigned)cdiv(W, SM), (unsigned)cdiv(r, SJ), (unsigned)pieces),
                     dim3(kThreads), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  int64_t blocks = cdiv(W * r, 4096);
  if (blocks > 256) blocks = 256;
  hipLaunchKernelGGL(multi_tn_reduce_kernel<RANKS_IN>, dim3((unsigned)blocks, (unsigned)A), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

bool multi_dense_supported(int64_t K, int64_t N, int r) {
  const int64_t rp = cdiv(r, 64) * 64, two_gb = (int64_t)1 << 31, np = cdiv(N, 64) * 64;
  return K * np * 2 < two_gb && N * rp * 2 < two_gb && K * rp * 2 < two_gb;
}

bool multi_forward_supported(int64_t M, int64_t K, int64_t N, int r) {
  return multi_small_fits(M, K, N) || multi_dense_supported(K, N, r);
}

// M <= 128: a single token or a few through the GEMVs where they apply, else
// the one-pass product.
static hipError_t multi_forward_small(const NF4View& W, const NF4Table& tab, const uint16_t* X, int64_t M,
                                      const MultiIds& mi, const uint16_t* L1, const uint16_t* L2, int r, uint16_t* Y,
                                      uint16_t* T_out, float* part, float* tpart, hipStream_t stream) {
  const int64_t K = W.cols, N = W.rows;
  if (gemv1_applies(W, M, r)) return launch_gemv1_multi(W, tab, X, mi, L1, L2, r, Y, T_out, tpart, stream);
  hipError_t e = launch_multi_small_t(X, M, K, mi, L1, r, tpart, stream);
  if (e != hipSuccess) return e;
  const int Z = multi_small_t_slices(K);
  if (gemv_multi_applies(W, M, r))
    return timed(kTimeGemv, stream,
                 [&] { return launch_gemv_multi(W, tab, X, M, mi, tpart, Z, L2, r, Y, T_out, stream); });
  return timed(kTimeMidGemm, stream, [&]() -> hipError_t {
    const hipError_t b = launch_multi_small_base(W, tab, X, M, part, stream);
    if (b != hipSuccess) return b;
    return launch_multi_small_finish(part, multi_small_slices(M, K, N), M, N, mi, tpart, Z, r, L2, Y, T_out, stream);
  });
}

hipError_t multi_forward(const NF4View& W, const NF4Table& tab, const uint16_t* X, int64_t M, const int32_t* ids,
                               int A, const uint16_t* L1, const uint16_t* L2, int r, const float* scale, uint16_t* Y,
                               uint16_t* T_out, void* ws, hipStream_t stream) {
  const int64_t K = W.cols, N = W.rows, segs = A < M ? A : M;
  const int rp = (int)cdiv(r, 64) * 64;
  const MultiWorkspace L = multi_workspace_layout(M, K, N, r, A, false);
  char* base = static_cast<char*>(ws);
  uint16_t* sT = reinterpret_cast<uint16_t*>(base + L.st_off);
  uint16_t* l2t = reinterpret_cast<uint16_t*>(base + L.b2_off);
  uint16_t* wd = reinterpret_cast<uint16_t*>(base + L.wd_off);
  int32_t* slot = reinterpret_cast<int32_t*>(base + L.slot_off);
  float* part = reinterpret_cast<float*>(base + L.part_off);
  if (multi_small_fits(M, K, N))
    return multi_forward_small(W, tab, X, M, MultiIds{ids, A, scale}, L1, L2, r, Y, T_out, part,
                               reinterpret_cast<float*>(base + L.tpart_off), stream);
  RouteView rv;
  hipError_t e = route(ids, M, A, base, L.perm_off, L.start_off, L.adapter_off, L.count_off, slot, &rv, stream);
  if (e != hipSuccess) return e;
  e = rows_by_adapter<true>(X, K, L1, 0, K * r, M, r, rp, A, ids, scale, rv, part, sT, T_out, stream);
  if (e != hipSuccess) return e;
  e = zero_words(sT + M * rp, rp * 2, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(multi_l2t_kernel, dim3((unsigned)cdiv(N, 64), (unsigned)(rp / 64), (unsigned)segs), dim3(256), 0,
                     stream, L2, N, r, rp, rv, l2t);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  e = launch_dequant_rows(W, tab, wd, stream);
  if (e != hipSuccess) return e;
  return gemm_by_adapter(X, K, wd, M, N, sT, l2t, rp, N * rp, slot, Y, ids, A, rv, base, L, kTimeFwdGemm, stream);
}

hipError_t multi_backward(const NF4View& W, const NF4Table& tab, const uint16_t* X, const uint16_t* dY, int64_t M,
                          const int32_t* ids, int A, const uint16_t* L1, const uint16_t* L2, int r, const float* scale,
                          const uint16_t* T, uint16_t* dX, void* dL1, void* dL2, bool grad_bf16, void* ws,
                          hipStream_t stream) {
  const int64_t K = W.cols, N = W.rows, segs = A < M ? A : M;
  const int64_t each = grad_bf16 ? 2 : 4;
  if (M == 0) {  // no rows: all gradients are zero
    const hipError_t e = zero_words(dL1, A * K * r * each, stream);
    return e == hipSuccess ? zero_words(dL2, A * N * r * each, stream) : e;
  }
  const int rp = (int)cdiv(r, 64) * 64;
  const MultiWorkspace L = multi_workspace_layout(M, K, N, r, A, true);
  char* base = static_cast<char*>(ws);
  uint16_t* sU = reinterpret_cast<uint16_t*>(base + L.st_off);
  int32_t* slot = reinterpret_cast<int32_t*>(base + L.slot_off);
  float* part = reinterpret_cast<float*>(base + L.part_off);
  RouteView rv;
  hipError_t e = route(ids, M, A, base, L.perm_off, L.start_off, L.adapter_off, L.count_off, slot, &rv, stream);
  if (e != hipSuccess) return e;
  e = rows_by_adapter<false>(dY, N, L2, N, N * r, M, r, rp, A, ids, scale, rv, part, sU, nullptr, stream);
  if (e != hipSuccess) return e;
  if (dX) {
    e = zero_words(sU + M * rp, rp * 2, stream);
    if (e != hipSuccess) return e;
    const uint16_t* b2 = L1;
    const bool padded = rp != r;
    if (padded) {
      uint16_t* l1p = reinterpret_cast<uint16_t*>(base + L.b2_off);
      hipLaunchKernelGGL(multi_l1p_kernel, dim3((unsigned)cdiv(K * rp / 8, 256), (unsigned)segs), dim3(256), 0, stream,
                         L1, K, r, rp, rv, l1p);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
      b2 = l1p;
    }
    // the GEMM reduces over whole stages of 64: pad a ragged N with zeros
    const int64_t np = cdiv(N, 64) * 64;
    const uint16_t* dYp = dY;
    if (np != N) {
      uint16_t* p = reinterpret_cast<uint16_t*>(base + L.dy_off);
      hipLaunchKernelGGL(multi_pad_rows_kernel, dim3(capped(cdiv(M * np / 8, 256))), dim3(256), 0, stream, dY, M, N, p,
                         np);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
      dYp = p;
    }
    uint16_t* wdt = reinterpret_cast<uint16_t*>(base + L.wd_off);
    e = launch_dequant_cols(W, tab, wdt, np, stream);
    if (e != hipSuccess) return e;
    e = gemm_by_adapter(dYp, np, wdt, M, K, sU, b2, rp, K * rp, padded ? slot : nullptr, dX, ids, A, rv, base, L,
                        kTimeDxGemm, stream);
    if (e != hipSuccess) return e;
  }
  if (!T) {
    uint16_t* t = reinterpret_cast<uint16_t*>(base + L.t_off);
    e = rows_by_adapter<true>(X, K, L1, 0, K * r, M, r, rp, A, ids, scale, rv, part, nullptr, t, stream);
    if (e != hipSuccess) return e;
    T = t;
  }
  e = gradient<true>(X, K, sU, rp, M, r, A, nullptr, rv, part, dL1, grad_bf16, stream);
  if (e != hipSuccess) return e;
  return gradient<false>(dY, N, T, r, M, r, A, scale, rv, part, dL2, grad_bf16, stream);
}

}  // namespace qlora
