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
//   small_base_kernel          the base product: K-slice partials (fp32) from
//                              one pass over the 4-bit weight; or, for few
//                              rows, the GEMV, which also adds the adapters
//                              (gemv.hip)
//   small_multi_finish_kernel  Y = bf16(the partials' sum + s_a T L2_a), for
//                              up to 16 rows of one adapter and 512 columns:
//                              an adapter's L2 is read once per 16 rows
// At these sizes the weight stream (0.52 B per weight) and the live adapters
// are all there is to read; the launches' latency is the rest. 96 rows of 24
// rank-16 adapters and of none, 4096 -> 11008: T 5.3 us, base 27.4, finish 8.2;
// the call 39 us. (In the finish, loading the base's first two slices before T's
// took 10.3 us: 186 registers leave two waves per SIMD.)
#include "common.h"
#include "launch.h"

#include <type_traits>

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

// ---- base product ------------------------------------------------------------------
//
// part[z][m][n] = sum over slice z of X[m][k] Wd[n][k], Wd = bf16(RN32(q[code] a')),
// M <= 32 MT. A workgroup owns 128 weight rows and one K-slice, in stages of
// 128 k; wave (wn, wk) of its 8 takes weight rows 64 wn .. +64 and the stage's
// 32 k from 32 wk with v_mfma_f32_32x32x16_bf16 (A = weights, B = X): two row
// groups share each X fragment that is read from LDS.
//   * Codes (8 KB per stage) and X (8 MT KB) come by direct copies into LDS
//     rings, X two stages ahead, the codes as far ahead as LDS allows. There is
//     no other load in the loop, so the counted waits before the stage
//     barriers are exact.
//   * The weights of a stage are dequantised among the MFMAs of the one before:
//     table reads, conversions and MFMAs of a wave overlap instead of
//     following each other in all waves at once.
//   * A lane dequantises its own A operands: 16 codes of each of its two rows,
//     in MFMA step s its codes 8 s .. 8 s + 8 (k = 16 (l/32) + 8 s + e: the X
//     operand uses the same k). So a weight is dequantised once for all M
//     columns, and one constant a' serves a row's whole stage.
//   * The constants of up to 16 stages are computed into LDS beforehand.
//   * The four k-parts of a workgroup are added through LDS at the end, from
//     where the partials are written in whole rows.
// Against 64-row workgroups with X staged through registers (the single
// adapter's one-pass kernel) X is read half as often from the L2 and the LDS
// reads per MFMA are half as many: M = 96, 4096 -> 11008 27.4 us (0.32 PFLOP/s,
// 0.8 TB/s of weights) against 47. A stage takes about 2600 clocks, where its
// MFMAs need 770, its LDS accesses 1200 and its dequantisation 1200 clocks of a
// SIMD: two waves per SIMD overlap them in part.
constexpr int kBaseThreads = 512;
constexpr int kBaseRows = 128;               // weight rows per workgroup
constexpr int kBaseK = 128;                  // k per stage
constexpr int kBaseStages = 3;
constexpr int kConstStages = 16;             // stages whose constants are in LDS at once
constexpr int kCodeBytes = kBaseRows * kBaseK / 2;

typedef __attribute__((address_space(3))) void lds_void_t;

// One 16-byte copy per lane into 1 KB of LDS (uniform base, the lane's 32-bit
// offset), not visible to the compiler: the caller waits for it with a counted
// vmcnt.
__device__ __forceinline__ void copy16(const char* from, uint32_t off, const void* lds) {
  const uint64_t v = reinterpret_cast<uint64_t>(from);   // scalar registers, also where the compiler sees no uniformity
  const uint64_t base = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v) |
                        (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32)) << 32;
  const uint32_t m0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void_t*)lds);
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" :: "v"(off), "s"(base), "s"(m0)
               : "memory", "m0");
}

// chunk c of 128-byte X row m sits at c ^ x_swz(m), chunk c of 64-byte code row
// n at c ^ c_swz(n): 16 consecutive rows' reads cover all banks, and rows 32
// apart have the same swizzle
__device__ __forceinline__ int x_swz(int m) { return (m >> 1) & 7; }
__device__ __forceinline__ int c_swz(int n) { return (n >> 2) & 3; }

template <int MT>
struct BaseLds {
  static constexpr int kXBytes = 2 * 32 * MT * 128;            // per stage: two 64-k halves of 32 MT rows
  static constexpr int kC = MT == 1 ? 4 : MT == 2 ? 8 : MT == 3 ? 6 : 5;   // code stages: what LDS leaves (two workgroups for MT = 1)
  static constexpr int kCodes = kBaseStages * kXBytes;
  static constexpr int kConst = kCodes + kC * kCodeBytes;      // fp32 [2 kConstStages][128]
  static constexpr int kOut = 2 * 32 * MT * (kBaseRows + 4) * 4;   // the k-parts' sums, over the rings
  static constexpr int kTotal = kConst + 2 * kConstStages * kBaseRows * 4;
  static_assert(kOut <= kConst, "the output tiles fit over the rings");
};

// RAGGED: K is an odd multiple of 64; the last stage is then compiled apart. A
// check in the loop of one variant for all took 0.4 to 1.5 us of every call (60
// rows 4096 -> 11008 35.2 -> 36.7); so it costs K = 4160 0.4 to 0.8 us (60 rows
// -> 11008 37.7 -> 38.2) and nothing where K is a multiple of 128.
// PAIR: weight blockIdx.z of two (of one shape), the second's partials behind the first's; from blockIdx.z = 2 on T's
// tg workgroups, which the base product does not wait for. 96 rows, 4096 -> 2 x 11008: 41.3 us, of tiles on 172 of the
// 256 CUs. T by a launch of its own before was slower, whole calls of 17 to 128 rows and ranks 16 to 256: 3 to 10 us
// where CUs are left idle, by the last round of tiles too (4096 -> 2 x 11008 96 rows rank 16 53.0 -> 49.1, 128 rows rank
// 256 120.7 -> 112.2; -> 2 x 22016 33 rows rank 16 82.5 -> 78.2). With none idle it is 0.2 to 1.8 us slower too, but for
// rank 256 of 96 and 128 rows, where it was 0.3 to 1.8 us faster in ten of twelve calls (-> 2 x 16384 161.5, here 162.5).
struct SecondBase {
  NF4View W;
  NF4Table tab;
  const uint16_t* L1;        // [2][K][r]
  float* t_part;             // [2][Z][M][r]
  int r, Z, tg;              // tg: 2 Z ranks' tiles of 64 rows' tiles of 16
};

// T's partials of 16 rows, 64 ranks and 512 k of one of two adapters, by 8 waves of 2 x 32 k each: those of
// small_t_partial_kernel but for the order of the waves' sum.
__device__ __forceinline__ void pair_t_body(const SecondBase& o, const uint16_t* __restrict__ X, int M, int64_t K, int id, float* red) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int jts = (o.r + 63) / 64, mtiles = (M + 15) / 16;
  const int z = id % o.Z, jt0 = id / o.Z % jts, mt = id / (o.Z * jts) % mtiles, w = id / (o.Z * jts * mtiles);
  const uint16_t* L1 = o.L1 + (int64_t)w * K * o.r;
  float* P = o.t_part + ((int64_t)w * o.Z + z) * M * o.r;
  const int row = lane & 15, j0 = 64 * jt0, mb = 16 * mt;
  u32x4_t xa[2];
  uint32_t h[2][4][8];                                 // all loads first (one round trip)
#pragma unroll
  for (int k2 = 0; k2 < 2; ++k2) {
    const int64_t kw = (int64_t)z * 512 + (2 * wave + k2) * 32 + 8 * (lane >> 4);
    xa[k2] = u32x4_t{0u, 0u, 0u, 0u};
    if (mb + row < M && kw < K) xa[k2] = *reinterpret_cast<const u32x4_t*>(X + (int64_t)(mb + row) * K + kw);  // K % 64 == 0
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      const int j = j0 + 16 * jt + row;
      const bool in = j < o.r && kw < K;
      const uint16_t* lp = L1 + (in ? kw * o.r + j : 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k2][jt][i] = lp[in ? (int64_t)i * o.r : 0];
      if (!in) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k2][jt][i] = 0u;
      }
    }
  }
#pragma unroll
  for (int jt = 0; jt < 4; ++jt) {
    f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k2 = 0; k2 < 2; ++k2) {
      const uint32_t* q = h[k2][jt];
      const u32x4_t b = {q[0] | (q[1] << 16), q[2] | (q[3] << 16), q[4] | (q[5] << 16), q[6] | (q[7] << 16)};
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, xa[k2]), __builtin_bit_cast(bf16x8_t, b), acc, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) red[(wave * 16 + 4 * (lane >> 4) + i) * 64 + 16 * jt + row] = acc[i];
  }
  __syncthreads();
#pragma unroll
  for (int m = wave; m < 16; m += 8) {                 // thread (m, lane) sums the waves in order
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < 8; ++q) v += red[(q * 16 + m) * 64 + lane];
    if (mb + m < M && j0 + lane < o.r) P[(int64_t)(mb + m) * o.r + j0 + lane] = v;
  }
}

template <int MT, bool RAGGED, bool PAIR>
__global__ __launch_bounds__(kBaseThreads) void small_base_kernel(NF4View W, NF4Table tab,
                                                                  const uint16_t* __restrict__ X, int M, int slice,
                                                                  float* __restrict__ part, SecondBase other) {
  using L = BaseLds<MT>;
  __shared__ float s_q[16];                            // a fixed address: table reads need no base
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  if constexpr (PAIR) {
    static_assert(kBaseThreads / 64 * 16 * 64 * 4 <= L::kTotal, "the sums of T's workgroups fit");
    if (blockIdx.z > 1) {                              // uniform
      const int n = (int)((gridDim.z - 2) * gridDim.y * gridDim.x);
      for (int id = (int)(((blockIdx.z - 2) * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x); id < other.tg; id += n) {
        pair_t_body(other, X, M, W.cols, id, reinterpret_cast<float*>(smem));
        __syncthreads();                               // the sums' LDS is written again
      }
      return;
    }
    if (blockIdx.z) {
      W = other.W;
      part += (int64_t)gridDim.y * M * W.rows;
    }
  }
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave & 1, wk = wave >> 1;
  const int64_t N = W.rows, K = W.cols;
  const int64_t n0 = (int64_t)blockIdx.x * kBaseRows;
  const int64_t k0 = (int64_t)blockIdx.y * slice;
  const int64_t k1 = k0 + slice < K ? k0 + slice : K;
  const int ns = (int)((k1 - k0 + kBaseK - 1) / kBaseK);
  float* s_a = reinterpret_cast<float*>(smem + L::kConst);
  if (tid < 16) s_q[tid] = PAIR && blockIdx.z ? other.tab.q[tid] : tab.q[tid];

  // Copies: waves 0-3 bring X, waves 4-7 the codes, each with a wait count of
  // its own (a wave's copies complete in order: codes, from HBM and several
  // stages ahead, would hold up X, from the L2 and two stages ahead).
  // Code instruction q of wave 4 + w: rows 16 (2 w + q) .. +16, lane -> row lane / 4, chunk lane % 4;
  // X instruction q of wave w: 8 rows of one half, lane -> row lane / 8, chunk lane % 8. Rows past N or M
  // repeat the last one; k past the slice (the second half of a last stage) reads its first half: the constants
  // there are 0, and X is cleared before it is used (0 times a copied infinity would be NaN). Stage numbers past
  // the last repeat its addresses: every stage issues the same number of copies, and their data is not used.
  constexpr int kXPer = 2 * MT, kCPer = 2;
  const bool brings_x = wave < 4;
  const char* base = brings_x ? reinterpret_cast<const char*>(X + k0) : reinterpret_cast<const char*>(W.codes + (n0 * K + k0) / 2);
  uint32_t off[kXPer], off_half[kXPer];                  // of a whole stage, and of one with 64 k only
#pragma unroll
  for (int q = 0; q < kXPer; ++q) {
    if (brings_x) {
      const int t = kXPer * wave + q;                    // 8 MT instructions: half t / (4 MT)
      const int rl = 8 * (t % (4 * MT)) + (lane >> 3);
      const uint32_t row = (uint32_t)(rl < M ? rl : M - 1) * (uint32_t)K;
      const uint32_t k = 8u * ((lane & 7) ^ x_swz(rl));
      off[q] = 2u * (row + 64u * (t / (4 * MT)) + k);
      off_half[q] = 2u * (row + k);
    } else {
      const int rl = 16 * (2 * (wave - 4) + (q & 1)) + (lane >> 2);
      const uint32_t row = (uint32_t)(n0 + rl < N ? rl : N - 1 - n0) * (uint32_t)(K / 2);
      const uint32_t c = (lane & 3) ^ c_swz(rl);
      off[q] = row + 16u * c;
      off_half[q] = row + 16u * (c & 1u);
    }
  }
  const bool ragged = RAGGED && k1 == K;                 // the last stage has 64 k
  // copies q0 .. q1 of the wave's share of X of stage st, and of the codes
  auto issue_x = [&](int st, int q0, int q1) {
    char* buf = smem + (st % kBaseStages) * L::kXBytes + kXPer * wave * 1024;
    const int at = st < ns ? st : ns - 1;
    const char* from = base + (int64_t)at * (2 * kBaseK);
    const bool h = ragged && at == ns - 1;
#pragma unroll
    for (int q = q0; q < q1; ++q) copy16(from, h ? off_half[q] : off[q], buf + q * 1024);
  };
  auto issue_c = [&](int st, int q0, int q1) {
    char* buf = smem + L::kCodes + (st % L::kC) * kCodeBytes + kCPer * (wave - 4) * 1024;
    const int at = st < ns ? st : ns - 1;
    const char* from = base + (int64_t)at * (kBaseK / 2);
    const bool h = ragged && at == ns - 1;
#pragma unroll
    for (int q = q0; q < q1; ++q) copy16(from, h ? off_half[q] : off[q], buf + q * 1024);
  };
  // constants of stages st0 .. st0 + kConstStages: [block][row]; lane -> block
  // of one row, so that a row's bytes are read together. All loads first, and
  // none under a branch: the compiler would wait for each where its branches
  // join (8 round trips to HBM).
  const bool dq = W.absmax32 == nullptr;
  const uint8_t* bytes = dq ? W.absmax8 : reinterpret_cast<const uint8_t*>(W.absmax32);
  const float* scales = dq ? W.scale2 : W.absmax32;
  const float mu = *(dq ? W.mean : W.absmax32);
  const int nblk = (int)(K / kBlock);
  auto constants = [&](int st0) {
    constexpr int kPer = 2 * kConstStages * kBaseRows / kBaseThreads;
    const int b = tid % (2 * kConstStages), row0 = tid / (2 * kConstStages);
    const int blk = (int)(k0 / kBlock) + 2 * st0 + b;
    const bool in = blk < (int)(k1 / kBlock);
    uint8_t c8[kPer];
    float sc[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t n = n0 + row0 + i * (kBaseRows / kPer);
      const int64_t at = (n < N ? n : N - 1) * nblk + (in ? blk : 0);
      c8[i] = bytes[dq ? at : 0];
      sc[i] = scales[dq ? at / kDqBlock : at];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float a = dq ? block_scale(c8[i], sc[i], mu) : sc[i];
      s_a[b * kBaseRows + row0 + i * (kBaseRows / kPer)] = in ? a : 0.0f;
    }
  };

  f32x16_t acc[2][MT];
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[g][t][v] = 0.0f;
  const int half = lane >> 5;
  const char* table = reinterpret_cast<const char*>(s_q);
  // lane offsets of the codes and constants of its row in row group g, and of
  // its X fragment in step s (column m = l%32; columns 32 t + l%32 follow 4 KB apart)
  uint32_t c_off[2], a_off[2], x_off[2];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int row = 64 * wn + 32 * g + (lane & 31);
    c_off[g] = (uint32_t)(row * 64 + ((wk ^ c_swz(row)) << 4) + 8 * half);
    a_off[g] = (uint32_t)((wk >> 1) * kBaseRows + row);
    x_off[g] = (uint32_t)((wk >> 1) * (32 * MT * 128) + (lane & 31) * 128 +
                          ((((wk & 1) * 4 + 2 * half + g) ^ x_swz(lane & 31)) << 4));
  }
  struct Codes {
    u32x2_t c[2];
    float a[2];
  };
  auto codes_of = [&](int st) {
    Codes d;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      d.c[g] = *reinterpret_cast<const u32x2_t*>(smem + L::kCodes + (st % L::kC) * kCodeBytes + c_off[g]);
      d.a[g] = s_a[2 * (st % kConstStages) * kBaseRows + a_off[g]];
    }
    return d;
  };
  // part p = 2 g + s of a stage's weights: row group g, step s; its 8 table values, then its A operand
  auto look = [&](const Codes& d, int p, float* f) {
    const uint32_t w = d.c[p >> 1][p & 1];
    const uint32_t lo = (w << 2) & 0x3C3C3C3Cu, hi = (w >> 2) & 0x3C3C3C3Cu;   // table offsets, a byte each
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = *reinterpret_cast<const float*>(table + ((lo >> (8 * e)) & 0xFFu));
      f[2 * e + 1] = *reinterpret_cast<const float*>(table + ((hi >> (8 * e)) & 0xFFu));
    }
  };
  auto convert = [&](const Codes& d, int p, const float* f) {
    const float a = d.a[p >> 1];
    return u32x4_t{pack_bf16x2(f[0] * a, f[1] * a), pack_bf16x2(f[2] * a, f[3] * a), pack_bf16x2(f[4] * a, f[5] * a),
                   pack_bf16x2(f[6] * a, f[7] * a)};
  };
  u32x4_t w0[4], w1[4];
  constants(0);
  if (brings_x) {
    issue_x(0, 0, kXPer);
    issue_x(1, 0, kXPer);
  } else {
#pragma unroll
    for (int s = 0; s < L::kC; ++s) issue_c(s, 0, kCPer);
    asm volatile("s_waitcnt vmcnt(%0)" :: "n"(kCPer * (L::kC - 1)) : "memory");   // the codes of stage 0
  }
  __syncthreads();
  {
    const Codes d = codes_of(0);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      float f[8];
      look(d, p, f);
      w0[p] = convert(d, p, f);
    }
  }
  // Stage st needs X of st and the codes of st + 1. Behind them may be in
  // flight: X of st + 1, the codes of st + 2 .. st + kC - 1. The buffer that the
  // codes of st + kC go to held those of st, read in the stage before. The
  // weights of st + 1 (past the last stage: not used) are made among the MFMAs
  // of st, part by part: the table reads of part p, the MFMAs of part p, the
  // conversion of part p - 1. The order is pinned: the scheduler would
  // otherwise gather all table reads before the first MFMA.
  auto stage = [&](int st, const u32x4_t* cur, u32x4_t* next, auto clear) {
    if ((st + 1) % kConstStages == 0 && st + 1 < ns) {  // uniform; long slices only: every wave has read stage st's
      __syncthreads();
      constants(st + 1);
    }
    if (brings_x) asm volatile("s_waitcnt vmcnt(%0)" :: "n"(kXPer) : "memory");
    else asm volatile("s_waitcnt vmcnt(%0)" :: "n"(kCPer * (L::kC - 2)) : "memory");
    __syncthreads();
    char* x = smem + (st % kBaseStages) * L::kXBytes;
    if constexpr (decltype(clear)::value) {               // every copy of this stage has landed
      for (int i = tid; i < 32 * MT * 128 / 16; i += kBaseThreads)
        reinterpret_cast<u32x4_t*>(x + 32 * MT * 128)[i] = u32x4_t{0u, 0u, 0u, 0u};
      __syncthreads();
    }
    const Codes d = codes_of(st + 1);
    bf16x8_t b[2][MT];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int t = 0; t < MT; ++t) b[s][t] = *reinterpret_cast<const bf16x8_t*>(x + x_off[s] + t * (32 * 128));
    __builtin_amdgcn_sched_barrier(0);
    float f[2][8];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      look(d, p, f[p & 1]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int t = 0; t < MT; ++t)
        acc[p >> 1][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, cur[p]), b[p & 1][t],
                                                                 acc[p >> 1][t], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      if (brings_x) issue_x(st + 2, p * kXPer / 4, (p + 1) * kXPer / 4);   // while the MFMAs run
      else issue_c(st + L::kC, p * kCPer / 4, (p + 1) * kCPer / 4);
      if (p > 0) next[p - 1] = convert(d, p - 1, f[(p - 1) & 1]);
      __builtin_amdgcn_sched_barrier(0);
    }
    next[3] = convert(d, 3, f[1]);
  };
  const std::false_type whole;
  const int n = ragged ? ns - 1 : ns;
  int st = 0;
  for (; st + 1 < n; st += 2) {
    stage(st, w0, w1, whole);
    stage(st + 1, w1, w0, whole);
  }
  if (st < n) {
    stage(st, w0, w1, whole);
#pragma unroll
    for (int p = 0; p < 4; ++p) w0[p] = w1[p];
  }
  if constexpr (RAGGED) {
    if (ragged) stage(n, w0, w1, std::true_type{});
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // no copy may land in the output tile
  // register v of lane l: weight row 64 wn + 32 g + (v%4) + 4 (l/32) + 8 (v/4), column m = 32 t + l%32
  constexpr int kPitch = kBaseRows + 4, kTile = 32 * MT * kPitch;
  float* out = reinterpret_cast<float*>(smem);
  __syncthreads();
#pragma unroll
  for (int h = 1; h >= 0; --h) {                        // k-parts 2, 3 into tiles 0, 1, then 0, 1 onto them
    if ((wk >> 1) == h) {
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x16_t& c = acc[g][t];
            f32x4_t* p = reinterpret_cast<f32x4_t*>(out + (wk & 1) * kTile + (32 * t + (lane & 31)) * kPitch + 64 * wn +
                                                   32 * g + 8 * q + 4 * half);
            f32x4_t v = {c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
            if (h == 0) v += *p;
            *p = v;
          }
    }
    __syncthreads();
  }
  for (int i = tid; i < M * (kBaseRows / 4); i += kBaseThreads) {
    const int m = i / (kBaseRows / 4), c = (i % (kBaseRows / 4)) * 4;
    const f32x4_t* p = reinterpret_cast<const f32x4_t*>(out + m * kPitch + c);
    if (n0 + c < N)                                    // N % 8 == 0
      *reinterpret_cast<f32x4_t*>(part + ((int64_t)blockIdx.y * M + m) * N + n0 + c) = p[0] + p[kTile / 4];
  }
}

// K-slices: as many workgroups as are resident at once (one or two per CU by
// LDS), in slices of whole stages; at most 8, whose sum in the finish costs what
// more would save here (whole call with 8 / 16: 24 rows 4096 -> 4096 18.8 / 22.4 us,
// 82 rows 5760 -> 1288 28.0 / 28.9, 121 rows 10432 -> 1104 42.6 / 40.5).
constexpr int kBaseTwoPerCu = 32;            // rows up to which two workgroups fit in a CU's LDS

struct BaseSplit {
  int slice, S;
};

BaseSplit base_split(int64_t M, int64_t K, int64_t N, int weights = 1) {
  const int64_t tiles = weights * ((N + kBaseRows - 1) / kBaseRows), steps = (K + kBaseK - 1) / kBaseK;
  const int64_t resident = (M <= kBaseTwoPerCu ? 2 : 1) * (int64_t)device_cu_count();
  int64_t S = resident / tiles;
  if (S > steps / 2) S = steps / 2;
  if (S > 8) S = 8;
  if (S < 1) S = 1;
  const int64_t per = (steps + S - 1) / S;
  return BaseSplit{(int)(per * kBaseK), (int)((steps + per - 1) / per)};
}

template <int MT, bool RAGGED, bool PAIR>
hipError_t run_base(const NF4View& W, const NF4Table& tab, const uint16_t* X, int M, const BaseSplit& sp, float* part,
                    const SecondBase& other, hipStream_t stream) {
  static bool attr_set = false;  // raise the dynamic-LDS limit once per instantiation (idempotent)
  if (!attr_set) {
    (void)hipFuncSetAttribute(reinterpret_cast<const void*>(&small_base_kernel<MT, RAGGED, PAIR>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, BaseLds<MT>::kTotal);
    (void)hipGetLastError();  // a refusal shows up as a launch error below
    attr_set = true;
  }
  const int64_t tiles = (W.rows + kBaseRows - 1) / kBaseRows;
  int64_t t_layers = (other.tg + tiles * sp.S - 1) / (tiles * sp.S);
  if (t_layers > 65533) t_layers = 65533;              // the grid's z is at most 65535
  const dim3 grid((unsigned)tiles, (unsigned)sp.S, PAIR ? 2 + (unsigned)t_layers : 1);
  hipLaunchKernelGGL((small_base_kernel<MT, RAGGED, PAIR>), grid, dim3(kBaseThreads), BaseLds<MT>::kTotal, stream, W, tab, X, M,
                     sp.slice, part, other);
  return hipGetLastError();
}

// ---- the sum ---------------------------------------------------------------------------

// Y = bf16(sum_z base[z][m][n] + sum_j bf16(s_a T[m][j]) L2_a[j][n]) for up to
// 16 rows of one group and 8 LANES columns, 8 per lane: a wave takes 64 / LANES
// rows at a time. The slices of T and of the base are added in order; workgroup
// column 0 writes T_out.
constexpr int kFinRank = 256;

template <int LANES>
__global__ __launch_bounds__(256) void small_multi_finish_kernel(const float* __restrict__ base, int S, int M, int N,
                                                                 const int32_t* __restrict__ ids, int A,
                                                                 const float* __restrict__ tpart, int Z, int r,
                                                                 const uint16_t* __restrict__ L2,
                                                                 const float* __restrict__ scale,
                                                                 uint16_t* __restrict__ Y,
                                                                 uint16_t* __restrict__ T_out) {
  __shared__ int rows[kGroup];
  constexpr int kPer = 64 / LANES, kQ = kGroup / (4 * kPer);   // rows per wave at a time, and times
  __shared__ float sT[kGroup][kFinRank + 4];          // rows of one wave in different banks
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const SmallGroup g = small_group<256>(ids, M, A, (int)blockIdx.y, rows);
  if (g.n == 0) return;                               // uniform
  const int n = (int)blockIdx.x * (8 * LANES) + 8 * (lane % LANES);
  const int first = wave * kPer;                      // row i of time q: first + lane / LANES + 4 kPer q
  const bool in = n < N;                              // N % 8 == 0
  const int nc = in ? n : 0;
  // L2 rows in batches; the first one's loads go out before anything waits
  constexpr int kBatch = 16;
  const uint16_t* B = L2 + (g.has ? (int64_t)g.a * r * N : 0) + nc;
  u32x4_t l2[kBatch];
  auto load_l2 = [&](int j0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      l2[u] = *reinterpret_cast<const u32x4_t*>(B + (int64_t)(j0 + u < r ? j0 + u : 0) * N);
  };
  load_l2(0);
  constexpr int kSlices = 4;
  float acc[kQ][8];
  int at[kQ];
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    at[q] = first + lane / LANES + 4 * kPer * q;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[q][e] = 0.0f;
    if (first + 4 * kPer * q >= g.n) continue;        // uniform per wave
    const float* p = base + (int64_t)rows[at[q] < g.n ? at[q] : 0] * N + nc;
    const int64_t pitch = (int64_t)M * N;
    for (int z = 0; z < S; z += kSlices) {            // that many slices' loads in flight, added in order
      f32x4_t a[kSlices], b[kSlices];
#pragma unroll
      for (int u = 0; u < kSlices; ++u) {
        const float* s = p + (z + u < S ? z + u : z) * pitch;
        a[u] = *reinterpret_cast<const f32x4_t*>(s);
        b[u] = *reinterpret_cast<const f32x4_t*>(s + 4);
      }
#pragma unroll
      for (int u = 0; u < kSlices; ++u) {
        if (z + u >= S) break;                        // uniform
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[q][e] += a[u][e];
          acc[q][4 + e] += b[u][e];
        }
      }
    }
  }
  if (g.has) {
    const float s = scale[g.a];
    for (int i = tid; i < g.n * r; i += 256) {
      const int k = i / r, j = i - k * r;
      const float* p = tpart + (int64_t)rows[k] * r + j;
      float v = 0.0f;
      for (int z = 0; z < Z; z += 8) {  // loads of 8 slices in flight, added in order
        float b[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) b[u] = p[(int64_t)(z + u < Z ? z + u : z) * M * r];
#pragma unroll
        for (int u = 0; u < 8; ++u) v += z + u < Z ? b[u] : 0.0f;
      }
      sT[k][j] = bf16_to_f32(f32_to_bf16(s * v));
      if (T_out && blockIdx.x == 0) T_out[(int64_t)rows[k] * r + j] = f32_to_bf16(v);
    }
  } else if (T_out && blockIdx.x == 0) {
    for (int i = tid; i < g.n * r; i += 256) T_out[(int64_t)rows[i / r] * r + i % r] = 0;
  }
  __syncthreads();
  if (g.has && first < g.n) {
    for (int j0 = 0; j0 < r; j0 += kBatch) {
      if (j0 > 0) load_l2(j0);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (j0 + u >= r) continue;
        const uint32_t v[4] = {l2[u].x, l2[u].y, l2[u].z, l2[u].w};
        float l[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          l[2 * e] = __uint_as_float(v[e] << 16);
          l[2 * e + 1] = __uint_as_float(v[e] & 0xFFFF0000u);
        }
#pragma unroll
        for (int q = 0; q < kQ; ++q) {
          if (first + 4 * kPer * q >= g.n) continue;
          const float t = sT[at[q]][j0 + u];          // rows past the group: not stored
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[q][e] = __builtin_fmaf(t, l[e], acc[q][e]);
        }
      }
    }
  }
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    if (at[q] < g.n && in)
      *reinterpret_cast<u32x4_t*>(Y + (int64_t)rows[at[q]] * N + n) =
          u32x4_t{pack_bf16x2(acc[q][0], acc[q][1]), pack_bf16x2(acc[q][2], acc[q][3]),
                  pack_bf16x2(acc[q][4], acc[q][5]), pack_bf16x2(acc[q][6], acc[q][7])};
  }
}

}  // namespace

int64_t multi_small_t_floats(int64_t M, int64_t K, int r) { return (K + kTK - 1) / kTK * M * r; }
int multi_small_t_slices(int64_t K) { return (int)((K + kTK - 1) / kTK); }

bool multi_small_fits(int64_t M, int64_t K, int64_t N) {
  return M >= 1 && M <= kMultiSmallRows && K < ((int64_t)1 << 23) && N <= ((int64_t)1 << 31) - 256;   // 32-bit offsets of 128 rows
}

int multi_small_slices(int64_t M, int64_t K, int64_t N) { return base_split(M, K, N).S; }

int64_t multi_small_partial_floats(int64_t M, int64_t K, int64_t N) {
  const int64_t few = M < kBaseTwoPerCu ? M : kBaseTwoPerCu;   // the slices depend on M only through this bound
  const int64_t a = base_split(few, K, N).S * few, b = base_split(M, K, N).S * M;
  return (a > b ? a : b) * N;
}

namespace {

template <bool PAIR>
hipError_t launch_base(const NF4View& W, const NF4Table& tab, const uint16_t* X, int64_t M, const BaseSplit& sp, float* part,
                       const SecondBase& other, hipStream_t stream) {
  auto run = [&](auto ragged) -> hipError_t {
    constexpr bool kRagged = decltype(ragged)::value;
    if (M <= 32) return run_base<1, kRagged, PAIR>(W, tab, X, (int)M, sp, part, other, stream);
    if (M <= 64) return run_base<2, kRagged, PAIR>(W, tab, X, (int)M, sp, part, other, stream);
    if (M <= 96) return run_base<3, kRagged, PAIR>(W, tab, X, (int)M, sp, part, other, stream);
    return run_base<4, kRagged, PAIR>(W, tab, X, (int)M, sp, part, other, stream);
  };
  return W.cols % kBaseK ? run(std::true_type{}) : run(std::false_type{});
}

}  // namespace

hipError_t launch_multi_small_base(const NF4View& W, const NF4Table& tab, const uint16_t* X, int64_t M, float* part,
                                   hipStream_t stream) {
  return launch_base<false>(W, tab, X, M, base_split(M, W.cols, W.rows), part, SecondBase{}, stream);
}

int small_pair_slices(int64_t M, int64_t K, int64_t N) { return base_split(M, K, N, 2).S; }

int64_t small_pair_partial_floats(int64_t M, int64_t K, int64_t N) {
  const int64_t few = M < kBaseTwoPerCu ? M : kBaseTwoPerCu;   // the slices depend on M only through this bound
  const int64_t a = base_split(few, K, N, 2).S * few, b = base_split(M, K, N, 2).S * M;
  return 2 * (a > b ? a : b) * N;
}

hipError_t launch_small_pair(const GatedBase& W, const uint16_t* X, int64_t M, const uint16_t* L1, int r, float* t_part, float* part,
                             hipStream_t stream) {
  const BaseSplit sp = base_split(M, W.gate.cols, W.gate.rows, 2);
  const int Z = small_t_slices(W.gate.cols);
  const SecondBase o{W.up, W.tab_up, L1, t_part, r, Z, (int)(2 * (int64_t)Z * ((r + 63) / 64) * ((M + 15) / 16))};
  return launch_base<true>(W.gate, W.tab_gate, X, M, sp, part, o, stream);
}

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
  // Workgroups of 512 columns, or of 128 where those would leave CUs idle: 34
  // rows of 8 rank-64 adapters 2944 -> 2392 26.2 instead of 39 us, 51 rows of one
  // 4608 -> 1128 23.0 / 33.9; 96 rows of 24, 4096 -> 11008 44.8 / 39.5.
  const int64_t groups = M < mi.A + 1 + M / kGroup ? M : mi.A + 1 + M / kGroup;   // at most
  if ((N + 511) / 512 * groups <= device_cu_count())
    hipLaunchKernelGGL(small_multi_finish_kernel<16>, dim3((unsigned)((N + 127) / 128), (unsigned)M), dim3(256), 0, stream,
                       base, S, (int)M, (int)N, mi.ids, mi.A, tpart, Z, r, L2, mi.scale, Y, T_out);
  else
    hipLaunchKernelGGL(small_multi_finish_kernel<64>, dim3((unsigned)((N + 511) / 512), (unsigned)M), dim3(256), 0, stream,
                       base, S, (int)M, (int)N, mi.ids, mi.A, tpart, Z, r, L2, mi.scale, Y, T_out);
  return hipGetLastError();
}

}  // namespace qlora
