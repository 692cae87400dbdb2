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
//   multi_prep_kernel    groups the rows by adapter (see multi.h) and, in its
//                        other workgroups, dequantises the weight
//   multi_nt_kernel      T = X L1_a and / or U = dY L2_a^T over 128-row pieces of
//                        the grouped rows, split over the reduction into fp32
//                        partials
//   multi_sum_kernel     sums them, scales each row by its s_a, rounds to bf16;
//                        its other workgroups lay out L2_a^T or L1_a for the GEMM
//   the dense GEMM       (dense_gemm.hip) walks the grouped rows; its adapter
//                        stages run over the segments that meet the tile
//   multi_tn_kernel      dL1_a and dL2_a: per piece of a segment, the products
//                        with the reduction down the rows
//   multi_finish_kernel  the sums over a segment's pieces, and the zeros of
//                        adapters without rows
// Launches with independent halves are one launch: at a few hundred rows each
// kernel takes 4 to 10 us, of which 2 to 4 are its start and end.
// Rows are gathered where a kernel loads them (a row's 128-byte stage slices
// are whole cache lines, so the gather costs no bandwidth), and every row
// buffer stays in the caller's order. All sums run in a fixed order.
//
// Measured, kernel times in us. The streaming kernels are bound by HBM, the GEMM
// by the matrix cores at the card's power limit:
//   4096 rows of 12 rank-64 adapters and of none, 4096 -> 11008, forward: prep
//   29 (113 MB, 3.9 TB/s), NT 14.4 (34 MB of X and its share of L1), sum 10.6, GEMM
//   360 (1.04 PFLOP/s); the call 370
//   8192 rows of 16, backward: prep 44 (113 MB, 2.6 TB/s), NT 54 (180 MB, 3.3
//   TB/s), sum 8.7, GEMM 588 (1.26 PFLOP/s), TN 84 (247 MB, 2.9 TB/s), finish
//   5.7; the call 744
//   391 rows of 4 rank-32 adapters, 4096 -> 4096, backward: prep 12, NT 7.4,
//   sum 6.1, GEMM 27 (0.49 PFLOP/s), TN 9.9, finish 5.4; the call 65
#include "common.h"
#include "dequant.h"
#include "launch.h"
#include "multi.h"

namespace qlora {

namespace {

typedef __attribute__((address_space(3))) void lds_void_t;

__device__ __attribute__((aligned(16))) uint32_t g_multi_zero[4];  // zero-initialised copy source

// ---- route ---------------------------------------------------------------------

constexpr int kRouteWaves = 4;

__device__ __forceinline__ int block_sum(int v, int* s) {   // 256 threads; s: kRouteWaves ints
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

struct RouteArgs {
  const int32_t* ids;
  int M, A;
  int32_t* perm;
  int32_t* start;
  int32_t* adapter;
  int32_t* count;
  int32_t* slot;          // an adapter's segment, where it has rows
  int32_t* bad;           // per segment: its adapter's laid-out operand has infinities or NaN
};

// Workgroup a < A: adapter a; workgroup A: the rows without one. Each reads
// all ids (from the L2 after the first): it counts the rows and the distinct
// adapters below its own, which are its place and its segment number, then
// writes its rows in order.
__device__ __forceinline__ void route_body(const RouteArgs& p, int a) {
  constexpr int kThreads = 64 * kRouteWaves;
  __shared__ uint32_t seen[kMultiMaxAdapters / 32];
  __shared__ int s_sum[kRouteWaves], s_wave[kRouteWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int M = p.M, A = p.A;
  const int words = (A + 31) / 32;
  for (int i = tid; i < words; i += kThreads) seen[i] = 0u;
  __syncthreads();
  int below = 0, mine = 0;
#pragma unroll 4
  for (int i = tid; i < M; i += kThreads) {
    const int v = p.ids[i];
    const bool has = v >= 0 && v < A;
    if (has && v < a) {
      ++below;
      atomicOr(&seen[v >> 5], 1u << (v & 31));      // the same bits in any order
    }
    mine += a < A ? v == a : !has;
  }
  below = block_sum(below, s_sum);
  mine = block_sum(mine, s_sum);             // its barriers also publish `seen`
  int rank = 0;
  for (int i = tid; i < words; i += kThreads) rank += __popc(seen[i]);
  rank = block_sum(rank, s_sum);
  if (tid == 0) {
    if (a == A) {
      p.count[0] = rank;
      p.start[rank] = below;
    } else if (mine > 0) {
      p.adapter[rank] = a;
      p.start[rank] = below;
      p.slot[a] = rank;
      p.bad[rank] = 0;
    }
  }
  if (mine == 0) return;                            // uniform
  int at = below;
  for (int i0 = 0; i0 < M; i0 += kThreads) {
    const int i = i0 + tid;
    const int v = i < M ? p.ids[i] : 0;
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
    if (take) p.perm[at + before + __popcll(b & ((1ull << lane) - 1ull))] = i;
    at += all;
  }
}

// Workgroups 0 .. A group the rows; the others dequantise the weight as stored
// (COLS = false) or transposed with rows of ldo (gx workgroups along k).
template <bool COLS>
__global__ __launch_bounds__(256) void multi_prep_kernel(RouteArgs p, NF4View W, NF4Table tab,
                                                         uint16_t* __restrict__ out, int64_t ldo, int gx) {
  const int b = (int)blockIdx.x - (p.A + 1);
  if (b < 0) {
    route_body(p, (int)blockIdx.x);
  } else if constexpr (COLS) {
    dequant_cols_body(W, tab, out, ldo, b % gx, b / gx);
  } else {
    dequant_rows_body(W, tab, out, b, (int)gridDim.x - (p.A + 1));
  }
}

// ---- adapter operands of the dense GEMM ---------------------------------------------

// Segments of small ranks share the 64 columns of a stage: rank r takes `width`
// columns (8, 16, 32, or whole stages), segment k the columns from
// (k % pack) width of group k / pack.
struct Packing {
  int width, pack;
};

__host__ __device__ inline Packing packing_of(int r) {
  const int w = r <= 8 ? 8 : r <= 16 ? 16 : r <= 32 ? 32 : (r + 63) / 64 * 64;
  return Packing{w, w < 64 ? 64 / w : 1};
}

struct LayArgs {
  const uint16_t* src;    // L2 [A][r][W] (transposed into [W][rp]) or L1 [A][W][r] (padded to [W][rp])
  uint16_t* out;          // per group [W][rp]; columns past a segment's r, and of segments that are none, zero
  int64_t W;
  int r, rp, blocks;      // blocks per group
  int32_t* bad;           // set where a segment has infinities or NaN; they are laid out as zeros
  bool transpose;
};

// Column c of group g's operand: its segment and rank (none: zeros).
struct LayColumn {
  int segment, rank;
  bool none;
};
__device__ __forceinline__ LayColumn lay_column(const LayArgs& p, const RouteView& rv, int g, int c) {
  const Packing pk = packing_of(p.r);
  const int s = c / pk.width, k = g * pk.pack + s, j = c - s * pk.width;
  return LayColumn{k, j, k >= rv.count[0] || j >= p.r};
}

// Eight values of segment k with infinities and NaN noted and zeroed.
__device__ __forceinline__ u32x4_t lay_finite(const LayArgs& p, int k, u32x4_t v) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool lo = (v[i] & 0x7F80u) == 0x7F80u, hi = (v[i] & 0x7F800000u) == 0x7F800000u;
    v[i] = (lo ? 0u : v[i] & 0xFFFFu) | (hi ? 0u : v[i] & 0xFFFF0000u);
    bad = bad || lo || hi;
  }
  if (bad) p.bad[k] = 1;                            // the same value from every thread
  return v;
}

// L2 of group g's segments transposed side by side: 64 output rows n and 64
// columns per workgroup, so that whole lines are written (one segment per
// workgroup: 13.3 against 6.7 us for 32 of rank 16, N = 11008).
__device__ __forceinline__ void lay_transposed(const LayArgs& p, const RouteView& rv, int g, int b) {
  __shared__ uint16_t tile[64][64 + 2];
  const int64_t N = p.W;
  const int tiles = p.rp / 64;
  const int64_t n0 = (int64_t)(b / tiles) * 64;
  const int j0 = (b % tiles) * 64;
  const int t = threadIdx.x;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int j = (t >> 3) + 32 * u, c = (t & 7) * 8;
    const LayColumn col = lay_column(p, rv, g, j0 + j);
    u32x4_t v = {0u, 0u, 0u, 0u};
    if (!col.none && n0 + c < N)
      v = lay_finite(p, col.segment, *reinterpret_cast<const u32x4_t*>(
              p.src + ((int64_t)rv.adapter[col.segment] * p.r + col.rank) * N + n0 + c));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) tile[c + e][j] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
  }
  __syncthreads();
  uint16_t* out = p.out + (int64_t)g * N * p.rp;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int n = (t >> 3) + 32 * u, c = (t & 7) * 8;
    if (n0 + n >= N) continue;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = (uint32_t)tile[n][c + 2 * e] | ((uint32_t)tile[n][c + 2 * e + 1] << 16);
    *reinterpret_cast<u32x4_t*>(out + (n0 + n) * p.rp + j0 + c) = u32x4_t{w[0], w[1], w[2], w[3]};
  }
}

// L1 of group g's segments side by side: 256 16-byte pieces per workgroup.
__device__ __forceinline__ void lay_padded(const LayArgs& p, const RouteView& rv, int g, int b) {
  const int64_t i = (int64_t)b * 256 + threadIdx.x;
  const int per = p.rp / 8;
  if (i >= p.W * per) return;
  const int64_t row = i / per;
  const int c = (int)(i - row * per) * 8;           // 8 columns are one segment's (r % 8 == 0)
  const LayColumn col = lay_column(p, rv, g, c);
  u32x4_t v = {0u, 0u, 0u, 0u};
  if (!col.none)
    v = lay_finite(p, col.segment, *reinterpret_cast<const u32x4_t*>(
            p.src + ((int64_t)rv.adapter[col.segment] * p.W + row) * p.r + col.rank));
  *reinterpret_cast<u32x4_t*>(p.out + ((int64_t)g * p.W + row) * p.rp + c) = v;
}

// ---- pieces shared by the two adapter products -----------------------------------------

constexpr int SK = 64;       // reduction per stage
constexpr int SJ = 64;       // ranks per tile
constexpr int SM = 128;      // rows (nt) or columns (tn) per tile
constexpr int kThreads = 256;

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

constexpr int kNtStages = 2;

struct NtLds {
  __attribute__((aligned(1024))) uint16_t a[kNtStages][SM * SK];
  __attribute__((aligned(1024))) uint16_t b[kNtStages][SJ * SK];
  int row[SM];
};

// C[z][m][j] = sum over slice z of A[m][i] B_a[j][i]: 128 grouped rows of one
// segment by 64 ranks; 4 waves of 32 rows; one stage's copies are in flight
// while another is multiplied, and three workgroups fit in a CU's LDS (with
// three stages two would: 4096 rows of 4096 18.1 us against 14.4). With BT the adapter's operand has its
// ranks contiguous (L1 as stored) and its fragments come through the LDS
// transpose read; without, its reduction is contiguous (L2 as stored).
template <bool BT>
__device__ __forceinline__ void nt_body(const NtArgs& p, int z, NtLds& lds) {
  auto& sA = lds.a;
  auto& sB = lds.b;
  auto& s_row = lds.row;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const RoutePiece pc = route_piece(p.rv, (int)blockIdx.y, SM);
  if (pc.hi <= pc.lo) return;                       // uniform: no barrier was reached
  const int j0 = (int)blockIdx.z * SJ;
  const int64_t z0 = (int64_t)z * p.split;
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
    const int buf = st % kNtStages;
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
  for (int s = 0; s < kNtStages - 1; ++s)
    if (s < ns) issue(s);
  for (int st = 0; st < ns; ++st) {
    const int buf = st % kNtStages;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (st + kNtStages - 1 < ns) issue(st + kNtStages - 1);
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
  float* C = p.C + (int64_t)z * p.M * p.rp;
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

// Slices z < zu: U = dY L2_a^T (arguments u); the others: T = X L1_a (t).
__global__ __launch_bounds__(kThreads) void multi_nt_kernel(NtArgs u, int zu, NtArgs t) {
  __shared__ NtLds lds;
  const int z = (int)blockIdx.x;
  if (z < zu) nt_body<false>(u, z, lds);
  else nt_body<true>(t, z - zu, lds);
}

// scaled [M + 1][rp] = bf16(s_a sum_z S[z]) in the columns of the row's segment,
// its other columns and the last row zero; plain [M][r] = bf16(sum_z P[z]).
// Either may be null. Partials [Z][M][rp]. Rows without an adapter are zero.
struct SumArgs {
  const float* S;
  const float* P;
  int Zs, Zp;
  int64_t M;
  int r, rp;
  const int32_t* ids;
  int A;
  const float* scale;
  const int32_t* slot;
  uint16_t* scaled;
  uint16_t* plain;
};

__device__ __forceinline__ f32x4_t sum_slices(const float* p, int Z, int64_t pitch) {
  f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
  int z = 0;
  for (; z + 4 <= Z; z += 4) {  // loads of 4 slices in flight, added in order
    f32x4_t q[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) q[u] = *reinterpret_cast<const f32x4_t*>(p + (int64_t)(z + u) * pitch);
#pragma unroll
    for (int u = 0; u < 4; ++u) v += q[u];
  }
  for (; z < Z; ++z) v += *reinterpret_cast<const f32x4_t*>(p + (int64_t)z * pitch);
  return v;
}

__device__ __forceinline__ u32x2_t pack4(const f32x4_t& v, float s) {
  return u32x2_t{pack_bf16x2(s * v.x, s * v.y), pack_bf16x2(s * v.z, s * v.w)};
}

// 4 columns per thread of workgroups below `blocks`; the others lay out the
// GEMM's adapter operand.
__global__ __launch_bounds__(256) void multi_sum_kernel(SumArgs p, int blocks, LayArgs lay, RouteView rv) {
  if ((int)blockIdx.x >= blocks) {
    const int b = (int)blockIdx.x - blocks, g = b / lay.blocks;
    if (g * packing_of(lay.r).pack >= rv.count[0]) return;  // uniform
    if (lay.transpose) lay_transposed(lay, rv, g, b - g * lay.blocks);
    else lay_padded(lay, rv, g, b - g * lay.blocks);
    return;
  }
  const int w4 = p.rp / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m = i / w4;
  const int j = (int)(i - m * w4) * 4;
  if (m > p.M) return;
  const int a = m < p.M ? p.ids[m] : -1;
  const bool has = a >= 0 && a < p.A;
  const f32x4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t pitch = p.M * p.rp, at = m * p.rp;
  if (p.scaled) {
    const Packing pk = packing_of(p.r);
    const int c = has ? j - p.slot[a] % pk.pack * pk.width : -1;   // 4 columns are inside a segment's, or all outside
    const bool in = c >= 0 && c < p.r;
    *reinterpret_cast<u32x2_t*>(p.scaled + at + j) =
        pack4(in ? sum_slices(p.S + at + c, p.Zs, pitch) : zero, in ? p.scale[a] : 0.0f);
  }
  if (p.plain && m < p.M && j < p.r)
    *reinterpret_cast<u32x2_t*>(p.plain + m * p.r + j) = pack4(has ? sum_slices(p.P + at + j, p.Zp, pitch) : zero, 1.0f);
}

struct TnArgs {
  const uint16_t* L;      // [M][ldl]: X or dY
  const uint16_t* S;      // [M][lds]: U or T, r columns used
  void* out;              // per adapter: [W][r] (RANKS_IN = true) or [r][W]
  float* part;            // per piece and rank tile: [W][64] or [64][W]
  const float* scale;     // factor per adapter, or null
  int64_t ldl, lds, W, slab;   // slab: floats per piece (all its rank tiles)
  int r, rows, ring;      // rows per piece, bytes of the ring
  bool packed;            // S holds a segment's ranks in its own columns
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
// Three stages, two workgroups per CU. With two stages and three workgroups the
// kernel took 73 instead of 86 us (8192 rows, 16 adapters) and 11.4 instead of
// 9.8 us (391 rows), but the whole backward call 747 instead of 750 us and 67.6
// instead of 67.0: at the larger size the card's power sets the call's time.
constexpr int kTnStages = 3;

// Dynamic LDS: the ring, then the piece's rows. The ring has the stages that a
// piece of `rows` rows has, and one where segments of one stage are expected
// (adapters enough for all rows at 64 each): then more workgroups fit in a CU,
// which hides what a short piece waits for. A longer piece is right with it too.
// 88 rows of 44 rank-8 adapters, 9280 -> 3776, 37.6 -> 23.7 us (with only the rows
// of a short piece copied and multiplied); 926 rows of 32 rank-120 adapters,
// 3264 -> 7360, 88 -> 54.
int tn_stages(int64_t rows, int64_t M, int64_t segs) {
  if (rows <= SK || M <= SK * segs) return 1;
  return rows <= 2 * SK ? 2 : kTnStages;
}
int tn_lds(int64_t rows, int stages) { return stages * kTnStageBytes + (int)(rows < kTnRows ? rows : kTnRows) * 4; }

template <bool RANKS_IN>
__device__ __forceinline__ void tn_body(const TnArgs& p, int bx, char* ring) {
  int* s_row = reinterpret_cast<int*>(ring + p.ring);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const RoutePiece pc = route_piece(p.rv, (int)blockIdx.z, p.rows);
  if (pc.hi <= pc.lo) return;                       // uniform: no barrier was reached
  const int64_t c0 = (int64_t)bx * SM;
  const int j0 = (int)blockIdx.y * SJ;
  const Packing pk = packing_of(p.r);
  const uint16_t* S = p.S + (p.packed ? pc.k % pk.pack * pk.width : 0);
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
  // a single stage: only the MFMA steps that have rows
  auto copy_stage = [&](int st, int end, char* buf) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (4 * (4 * wave + i) >= end) continue;        // uniform
      const int m = st * SK + 4 * (4 * wave + i) + (lane >> 4);
      copy16(m < n ? reinterpret_cast<const char*>(p.L + (int64_t)s_row[m < n ? m : 0] * p.ldl + l_col[i]) : zero,
             buf + (4 * wave + i) * 1024);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (8 * (2 * wave + i) >= end) continue;
      const int m = st * SK + 8 * (2 * wave + i) + (lane >> 3);
      copy16(m < n && s_in[i] ? reinterpret_cast<const char*>(S + (int64_t)s_row[m < n ? m : 0] * p.lds + s_col[i]) : zero,
             buf + kTnLBytes + (2 * wave + i) * 1024);
    }
  };
  auto issue = [&](int st, int end) { copy_stage(st, end, ring + (st % kTnStages) * kTnStageBytes); };

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
  auto multiply = [&](const char* buf, int kk) {
    const int r0 = 16 * kk + rb;
    const bf16x8_t l = frag_tr(l_at(buf, r0), l_at(buf, r0 + 4));
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const bf16x8_t s = frag_tr(s_at(buf, r0, t), s_at(buf, r0 + 4, t));
      acc[t] = RANKS_IN ? __builtin_amdgcn_mfma_f32_32x32x16_bf16(l, s, acc[t], 0, 0, 0)
                        : __builtin_amdgcn_mfma_f32_32x32x16_bf16(s, l, acc[t], 0, 0, 0);
    }
  };
  if (p.ring == kTnStageBytes) {                    // one stage in LDS
    for (int st = 0; st < ns; ++st) {
      const int left = n - st * SK, end = left < SK ? (left + 15) & ~15 : SK;
      if (st > 0) __syncthreads();                  // the stage before has been read
      copy_stage(st, end, ring);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      for (int kk = 0; 16 * kk < end; ++kk) multiply(ring, kk);
    }
  } else if (ns == 1) {
    issue(0, (n + 15) & ~15);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    for (int kk = 0; 16 * kk < n; ++kk) multiply(ring, kk);
  } else {
#pragma unroll
    for (int s = 0; s < kTnStages - 1; ++s)
      if (s < ns) issue(s, SK);
    for (int st = 0; st < ns; ++st) {
      if (st + 1 < ns) asm volatile("s_waitcnt vmcnt(6)" ::: "memory");   // the next stage's 6 copies may stay in flight
      else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      if (st + kTnStages - 1 < ns) issue(st + kTnStages - 1, SK);
      const char* buf = ring + (st % kTnStages) * kTnStageBytes;
#pragma unroll
      for (int kk = 0; kk < SK / 16; ++kk) multiply(buf, kk);
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

// Planes below z1: the pieces; column tiles below x1: dL1 (arguments g1), the
// others: dL2 (g2). The planes from z1 on add the slices of a split dX: alone
// that was a launch of 5.8 us after the GEMM (391 rows of 4096).
__global__ __launch_bounds__(kThreads) void multi_tn_kernel(TnArgs g1, int x1, TnArgs g2, int z1, SplitSum sum) {
  extern __shared__ __attribute__((aligned(1024))) char tn_smem[];
  const int x = (int)blockIdx.x;
  if ((int)blockIdx.z >= z1) {
    const int64_t plane = (int64_t)gridDim.x * gridDim.y;
    const int64_t b = ((int64_t)blockIdx.z - z1) * plane + (int64_t)blockIdx.y * gridDim.x + x;
    split_sum_body(sum, b * kThreads + threadIdx.x);
    return;
  }
  if (x < x1) tn_body<true>(g1, x, tn_smem);
  else tn_body<false>(g2, x - x1, tn_smem);
}

// The gradients that multi_tn_kernel left open: the sums of a segment's
// several pieces, in order, and zeros for adapters without rows. Workgroup bx
// of `blocks` for adapter blockIdx.y; 4 consecutive values per thread and step.
template <bool RANKS_IN>
__device__ __forceinline__ void finish_body(const TnArgs& p, int bx, int blocks) {
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
  const float f = pieces > 0 && p.scale ? p.scale[a] : 1.0f;   // not times the zeros: an idle adapter's scale may be anything
  const int64_t total = p.W * p.r;                  // r % 8 == 0, W % 8 == 0: 4 values never leave a row
  for (int64_t i = ((int64_t)bx * 256 + threadIdx.x) * 4; i < total; i += (int64_t)blocks * 1024) {
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

__global__ __launch_bounds__(256) void multi_finish_kernel(TnArgs g1, int x1, TnArgs g2) {
  const int x = (int)blockIdx.x;
  if (x < x1) finish_body<true>(g1, x, x1);
  else finish_body<false>(g2, x - x1, (int)gridDim.x - x1);
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
// Workgroups per adapter of multi_finish_kernel: 4 values per thread, a few steps.
int finish_blocks(int64_t values) { return (int)(cdiv(values, 4096) < 128 ? cdiv(values, 4096) : 128); }
unsigned capped(int64_t blocks) { return (unsigned)(blocks < 1 ? 1 : blocks > 16384 ? 16384 : blocks); }

// Reduction slices of the NT products: about two workgroups per CU, from five
// slices on in eights: consecutive workgroups run on the 8 XCDs in turn, and
// then an XCD's L2 holds one slice of the adapters' operands instead of all
// (dY of 8192 x 11008, 16 adapters: 61.9 -> 58.9 us; X of 4096 x 4096: 15.9 -> 14.4).
struct NtSplit {
  int64_t len;
  int Z;
};
NtSplit nt_split(int64_t M, int64_t len, int A, int rp) {
  int64_t tiles = (cdiv(M, SM) + (A < M ? A : M) / 2) * (rp / SJ);
  if (tiles < 1) tiles = 1;
  const int64_t steps = cdiv(len, SK);
  int64_t z = 2 * (int64_t)device_cu_count() / tiles;
  if (z > 4) z = z > 8 ? 16 : 8;
  if (z > steps) z = steps;
  if (z < 1) z = 1;
  const int64_t per = cdiv(steps, z);
  return NtSplit{per * SK, (int)cdiv(steps, per)};
}

// The most rows times slices of nt_split for any batch of up to M rows: z
// slices are taken for at most 2 CUs / `least` tiles.
int64_t nt_partial_rows(int64_t M, int64_t len, int rp) {
  struct Slices {
    int64_t z, least;
  };
  int64_t most = M;
  for (const Slices& s : {Slices{16, 9}, Slices{8, 5}, Slices{4, 4}, Slices{3, 3}, Slices{2, 2}}) {
    const int64_t rows = 2 * (int64_t)device_cu_count() / (s.least * (rp / SJ)) * SM;
    const int64_t z = s.z < cdiv(len, SK) ? s.z : cdiv(len, SK), v = z * (rows < M ? rows : M);
    if (v > most) most = v;
  }
  return most;
}

// Pieces of the TN products that fill the device (128 columns of dL1 or dL2 per workgroup).
int64_t tn_wanted(int64_t K, int64_t N, int r) {
  const int64_t tiles = (cdiv(K, SM) + cdiv(N, SM)) * cdiv(r, SJ);
  return cdiv(2 * (int64_t)device_cu_count(), tiles);
}

// Rows per piece: whole segments up to kTnRows rows, so that most gradients are
// written once; fewer when the launch would not fill the device.
constexpr int kTnLeast = 256;

int tn_rows(int64_t M, int64_t K, int64_t N, int r) {
  int64_t rows = cdiv(cdiv(M, tn_wanted(K, N, r)), SK) * SK;
  if (rows > kTnRows) rows = kTnRows;
  if (rows < kTnLeast) rows = kTnLeast;
  return (int)rows;
}

// Partials of dL1 or dL2 for any batch of up to M rows: at most M / rows + the
// segments, none where every segment is one piece.
int64_t tn_part_floats(int64_t M, int64_t K, int64_t N, int64_t W, int r, int A) {
  const int64_t want = tn_wanted(K, N, r);
  if (M <= (want > 1 ? kTnLeast : kTnRows)) return 0;
  int64_t pieces = want > M / kTnRows ? want : M / kTnRows;
  if (pieces > M / kTnLeast) pieces = M / kTnLeast;
  return (pieces + (A < M ? A : M)) * W * cdiv(r, SJ) * SJ;
}

}  // namespace

// No part is smaller for more rows, so that a workspace for the largest batch
// serves the smaller ones too.
MultiWorkspace multi_workspace_layout(int64_t M, int64_t K, int64_t N, int r, int A, bool bwd) {
  MultiWorkspace L = {};
  if (!bwd && (M < 1 || multi_small_fits(M, K, N))) {   // the small paths
    L.part_off = 0;
    L.tpart_off = align_up((size_t)multi_small_partial_floats(M, K, N) * 4, 256);
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
  L.bad_off = take(segs * 4);
  L.st_off = take((M + 1) * rp * 2);   // s T or s U, and a row of zeros
  L.t_off = take(bwd ? M * r * 2 : 0);
  const int64_t groups = cdiv(segs, packing_of(r).pack);
  const int64_t wide = bwd ? groups * K * rp * 2 : groups * N * rp * 2;
  L.b2_off = take(wide);
  L.wd_off = take(K * np * 2);
  L.dy_off = take(bwd && N % 64 ? M * np * 2 : 0);
  int64_t part = nt_partial_rows(M, K, (int)rp) * rp;   // T's, then U's; then dL1's and dL2's, or the forward GEMM's
  if (bwd) {
    part += nt_partial_rows(M, N, (int)rp) * rp;
    const int64_t grads = tn_part_floats(M, K, N, K, r, A) + tn_part_floats(M, K, N, N, r, A);
    if (grads > part) part = grads;
  }
  if (!bwd) {
    const int64_t gemm = (int64_t)gemm_multi_partial_bytes(M, N, K) / 4;
    if (gemm > part) part = gemm;
  }
  L.part_off = take(part * 4);
  L.gpart_off = take(bwd ? (int64_t)gemm_multi_partial_bytes(M, K, np) : 0);   // dX's, added while dL1 and dL2 are computed
  L.total = off;
  if (!bwd && multi_small_fits(kMultiSmallRows, K, N)) {
    const size_t small = multi_workspace_layout(kMultiSmallRows, K, N, r, A, false).total;
    if (small > L.total) L.total = small;
  }
  return L;
}

namespace {

RouteArgs route_args(const int32_t* ids, int64_t M, int A, char* ws, const MultiWorkspace& L) {
  RouteArgs p;
  p.ids = ids;
  p.M = (int)M;
  p.A = A;
  p.perm = reinterpret_cast<int32_t*>(ws + L.perm_off);
  p.start = reinterpret_cast<int32_t*>(ws + L.start_off);
  p.adapter = reinterpret_cast<int32_t*>(ws + L.adapter_off);
  p.count = reinterpret_cast<int32_t*>(ws + L.count_off);
  p.slot = reinterpret_cast<int32_t*>(ws + L.slot_off);
  p.bad = reinterpret_cast<int32_t*>(ws + L.bad_off);
  return p;
}

RouteView view_of(const RouteArgs& p) { return RouteView{p.perm, p.start, p.adapter, p.count}; }

// Arguments of T = X L1_a (b_t) or U = dY L2_a^T over rows of `len` values.
NtArgs nt_args(const uint16_t* rows, int64_t len, const uint16_t* B, int64_t b_stride, int64_t M, int r, int rp,
               const NtSplit& sp, const RouteView& rv, float* part) {
  NtArgs a;
  a.A = rows; a.B = B; a.C = part;
  a.lda = len; a.ldb = len; a.b_stride = b_stride;
  a.M = M; a.len = len; a.split = sp.len;
  a.r = r; a.rp = rp; a.rv = rv;
  return a;
}

hipError_t launch_nt(const NtArgs* u, int zu, const NtArgs* t, int zt, int64_t M, int A, hipStream_t stream) {
  const NtArgs& any = u ? *u : *t;
  const int64_t pieces = M / SM + (A < M ? A : M);
  hipLaunchKernelGGL(multi_nt_kernel, dim3((unsigned)(zu + zt), (unsigned)pieces, (unsigned)(any.rp / SJ)),
                     dim3(kThreads), 0, stream, u ? *u : any, zu, t ? *t : any);
  return hipGetLastError();
}

// Workgroups of multi_sum_kernel: the sums, and the layout of one group's operand.
int64_t sum_blocks(int64_t M, int64_t rp) { return cdiv((M + 1) * rp / 4, 256); }
int64_t lay_blocks(int64_t W, int64_t rp, bool transpose) { return transpose ? cdiv(W, 64) * (rp / 64) : cdiv(W * rp / 8, 256); }

hipError_t launch_sum(const SumArgs& s, const LayArgs& lay, int64_t segs, const RouteView& rv, hipStream_t stream) {
  const int64_t blocks = sum_blocks(s.M, s.rp);
  const int64_t groups = cdiv(segs, packing_of(lay.r).pack);
  hipLaunchKernelGGL(multi_sum_kernel, dim3((unsigned)(blocks + groups * lay.blocks)), dim3(256), 0, stream, s, (int)blocks,
                     lay, rv);
  return hipGetLastError();
}

hipError_t zero_words(void* p, int64_t bytes, hipStream_t stream) {
  hipLaunchKernelGGL(multi_zero_kernel, dim3(capped(cdiv(bytes / 4, 256))), dim3(256), 0, stream,
                     static_cast<uint32_t*>(p), bytes / 4);
  return hipGetLastError();
}

TnArgs tn_args(const uint16_t* L, int64_t W, const uint16_t* S, int64_t lds, bool packed, int r, int rows, int ring,
               const float* scale, const RouteView& rv, float* part, void* out, bool out_bf16) {
  TnArgs a;
  a.L = L; a.S = S; a.out = out; a.part = part; a.scale = scale;
  a.ldl = W; a.lds = lds; a.W = W;
  a.slab = W * cdiv(r, SJ) * SJ;
  a.r = r;
  a.rows = rows;
  a.ring = ring;
  a.packed = packed;
  a.out_bf16 = out_bf16;
  a.rv = rv;
  return a;
}

}  // namespace

bool multi_dense_supported(int64_t K, int64_t N, int r) {
  const int64_t rp = cdiv(r, 64) * 64, two_gb = (int64_t)1 << 31, np = cdiv(N, 64) * 64;
  return K * np * 2 < two_gb && N * rp * 2 < two_gb && K * rp * 2 < two_gb;
}

bool multi_lay_supported(int64_t M, int64_t W, int r, int A, bool transpose) {
  const int64_t rp = cdiv(r, 64) * 64, groups = cdiv(A < M ? A : M, packing_of(r).pack);
  return sum_blocks(M, rp) + groups * lay_blocks(W, rp, transpose) < (int64_t)1 << 24;
}

bool multi_forward_supported(int64_t M, int64_t K, int64_t N, int r, int A) {
  return multi_small_fits(M, K, N) || (multi_dense_supported(K, N, r) && multi_lay_supported(M, N, r, A, true));
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
  float* part = reinterpret_cast<float*>(base + L.part_off);
  if (multi_small_fits(M, K, N))
    return multi_forward_small(W, tab, X, M, MultiIds{ids, A, scale}, L1, L2, r, Y, T_out, part,
                               reinterpret_cast<float*>(base + L.tpart_off), stream);
  const RouteArgs ra = route_args(ids, M, A, base, L);
  const RouteView rv = view_of(ra);
  hipLaunchKernelGGL(multi_prep_kernel<false>, dim3((unsigned)(A + 1 + dequant_rows_blocks(W))), dim3(256), 0, stream, ra,
                     W, tab, wd, (int64_t)0, 1);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const NtSplit sp = nt_split(M, K, A, rp);
  const NtArgs t = nt_args(X, K, L1, K * r, M, r, rp, sp, rv, part);
  e = launch_nt(nullptr, 0, &t, sp.Z, M, A, stream);
  if (e != hipSuccess) return e;
  const SumArgs s{part, part, sp.Z, sp.Z, M, r, rp, ids, A, scale, ra.slot, sT, T_out};
  const LayArgs lay{L2, l2t, N, r, rp, (int)lay_blocks(N, rp, true), ra.bad, true};
  e = launch_sum(s, lay, segs, rv, stream);
  if (e != hipSuccess) return e;
  const MultiSlab slab{rv, packing_of(r).pack, M, N * rp, ra.bad, L2, N * r, 1, N, r, packing_of(r).width};
  return timed(kTimeFwdGemm, stream,
               [&] { return launch_gemm_nt_multi(X, K, wd, K, M, N, K, sT, l2t, rp, slab, Y, part, nullptr, stream); });
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
  float* part = reinterpret_cast<float*>(base + L.part_off);
  const RouteArgs ra = route_args(ids, M, A, base, L);
  const RouteView rv = view_of(ra);
  // the GEMM reduces over whole stages of 64: a ragged N is padded with zeros
  const int64_t np = cdiv(N, 64) * 64;
  uint16_t* wdt = reinterpret_cast<uint16_t*>(base + L.wd_off);
  const int gx = (int)cdiv(K, 128);
  const int64_t dequant_blocks = dX ? gx * cdiv(np, 128) : 0;
  hipLaunchKernelGGL(multi_prep_kernel<true>, dim3((unsigned)(A + 1 + dequant_blocks)), dim3(256), 0, stream, ra, W, tab,
                     wdt, np, gx);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;

  const NtSplit su = nt_split(M, N, A, rp), st = nt_split(M, K, A, rp);
  float* upart = part + (int64_t)st.Z * M * rp;
  const NtArgs u = nt_args(dY, N, L2, N * r, M, r, rp, su, rv, upart), t = nt_args(X, K, L1, K * r, M, r, rp, st, rv, part);
  e = launch_nt(&u, su.Z, T ? nullptr : &t, T ? 0 : st.Z, M, A, stream);
  if (e != hipSuccess) return e;
  uint16_t* tbuf = T ? nullptr : reinterpret_cast<uint16_t*>(base + L.t_off);
  uint16_t* l1p = reinterpret_cast<uint16_t*>(base + L.b2_off);
  const SumArgs s{upart, part, su.Z, st.Z, M, r, rp, ids, A, scale, ra.slot, sU, tbuf};
  const LayArgs lay{L1, l1p, K, r, rp, (int)lay_blocks(K, rp, false), ra.bad, false};
  e = launch_sum(s, lay, dX ? segs : 0, rv, stream);
  if (e != hipSuccess) return e;
  if (!T) T = tbuf;

  SplitSum sum{nullptr, nullptr, 0, 0};
  if (dX) {
    float* gpart = reinterpret_cast<float*>(base + L.gpart_off);
    const uint16_t* dYp = dY;
    if (np != N) {
      uint16_t* p = reinterpret_cast<uint16_t*>(base + L.dy_off);
      hipLaunchKernelGGL(multi_pad_rows_kernel, dim3(capped(cdiv(M * np / 8, 256))), dim3(256), 0, stream, dY, M, N, p,
                         np);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
      dYp = p;
    }
    const MultiSlab slab{rv, packing_of(r).pack, M, K * rp, ra.bad, L1, K * r, r, 1, r, packing_of(r).width};
    e = timed(kTimeDxGemm, stream, [&] {
      return launch_gemm_nt_multi(dYp, np, wdt, np, M, K, np, sU, l1p, rp, slab, dX, gpart, &sum, stream);
    });
    if (e != hipSuccess) return e;
  }

  const int rows = tn_rows(M, K, N, r);
  float* part2 = part + tn_part_floats(M, K, N, K, r, A);
  const int64_t most = M < rows ? M : rows;          // rows of a piece
  const int ring = tn_stages(most, M, segs) * kTnStageBytes;
  const TnArgs g1 = tn_args(X, K, sU, rp, true, r, rows, ring, nullptr, rv, part, dL1, grad_bf16);
  const TnArgs g2 = tn_args(dY, N, T, r, false, r, rows, ring, scale, rv, part2, dL2, grad_bf16);
  const int64_t pieces = M / rows + segs, tiles = cdiv(K, SM) + cdiv(N, SM);
  const int64_t planes = cdiv(sum.values / 8, kThreads * tiles * cdiv(r, SJ));
  const dim3 grid((unsigned)tiles, (unsigned)cdiv(r, SJ), (unsigned)(pieces + planes));
  static bool attr_set = false;  // raise the dynamic-LDS limit once (idempotent)
  if (!attr_set) {
    (void)hipFuncSetAttribute(reinterpret_cast<const void*>(&multi_tn_kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                              tn_lds(kTnRows, kTnStages));
    (void)hipGetLastError();  // a refusal shows up as a launch error below
    attr_set = true;
  }
  hipLaunchKernelGGL(multi_tn_kernel, grid, dim3(kThreads), tn_lds(most, ring / kTnStageBytes), stream, g1, (int)cdiv(K, SM), g2, (int)pieces, sum);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int b1 = finish_blocks(K * r), b2 = finish_blocks(N * r);
  hipLaunchKernelGGL(multi_finish_kernel, dim3((unsigned)(b1 + b2), (unsigned)A), dim3(256), 0, stream, g1, b1, g2);
  return hipGetLastError();
}

}  // namespace qlora
