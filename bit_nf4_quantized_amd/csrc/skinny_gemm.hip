// Skinny adapter products of the QLoRA linear on gfx950 (rank r <= 64):
//
//   forward   T   = X L1           [M][r]   (reduction over K)
//   backward  U   = dY L2^T        [M][r]   (reduction over N)
//             dL1 = s X^T U        [K][r]   (reduction over the M tokens)
//             dL2 = s (X L1)^T dY  [r][N]   (reduction over the M tokens)
//
// (QLoRA pages, diycv.top, section 问题背景 LoRA equation and section
// 关键公式.) Each product reads one large activation (X or dY, 64-180 MB at
// 8192 tokens) once and a small rank-r operand, so it is HBM-bound; the
// kernels stream the large operand with coalesced 16-byte loads, keep the
// whole rank dimension (padded to 64) in one tile, and use
// v_mfma_f32_32x32x16_bf16 for the products. The reduction is split over
// blockIdx.z into fp32 partials that skinny_reduce_kernel sums in a fixed
// order, so results are deterministic.
//
// skinny_nt_kernel:  C[z][m][j] = sum_{k in slice z} A[m][k] B[j][k]
//   A [M][K] and B [64][K] (rows j >= r are zero) are both K-contiguous and
//   are copied global -> LDS by global_load_lds_dwordx4; 128 rows x 64 j per
//   workgroup, 4 waves of 32 rows, K-stages of 64, 3-stage ring. With LoRA
//   dropout (DROP) A is the adapter input X, and every A fragment is
//   dropped in registers after its LDS read (each A element is read by
//   exactly one lane), from the Philox words of its element indices.
// skinny_tn_dma_kernel:  C[z][c][j] = sum_{m in slice z} L[m][c] S[m][j]
//   the reduction runs down the rows of both operands; both are copied
//   global -> LDS in their memory layout into a 3-stage ring, and the MFMA
//   fragments (consecutive m of one column) are read with the LDS transpose
//   read; 128 columns c x 64 j per workgroup, M-stages of 64.
// skinny_tn_kernel<true>:  the same product with LoRA dropout on the large
//   operand (the adapter input X): each thread loads two rows x 8 columns,
//   drops them in registers from the Philox words of their element indices
//   m W + c, and writes them to LDS transposed as (m, m+1) pairs, so the
//   dropped copy of X is never written to memory.
#include "common.h"
#include "launch.h"
#include "philox.h"

namespace qlora {

namespace {

typedef __attribute__((address_space(3))) void lds_void_t;
typedef const __attribute__((address_space(1))) void gbl_void_t;

constexpr int SK = 64;     // reduction per stage (elements)
constexpr int SJ = 64;     // rank columns per tile (r padded)
constexpr int SM = 128;    // large-operand rows (nt) or columns (tn) per tile
constexpr int kSkThreads = 256;

// 16-byte chunk c of LDS row `row` lives at c ^ sk_swz(row): (row >> 1) keeps
// the fragment reads of 16 consecutive rows on distinct bank groups, and
// (row >> 4) separates the rows that 8 neighbouring threads write at the
// same reduction index when a tile is transposed into LDS.
__device__ __forceinline__ int sk_swz(int row) { return ((row >> 1) ^ (row >> 4)) & 7; }
__device__ __forceinline__ int sk_off(int row, int chunk) { return row * SK + ((chunk ^ sk_swz(row)) << 3); }

// ---- NT: both operands contiguous in the reduction -----------------------------

constexpr int kNtStages = 3;

struct NtArgs {
  const uint16_t* A;  // [M][lda]
  const uint16_t* B;  // [SJ][ldb]  (64 rows; rows >= r zero)
  float* C;           // [Z][M][SJ]
  int64_t lda, ldb, M, K, k_split;
  uint32_t thr;       // DROP: keep iff the element's Philox word >= thr; kept values scaled by c
  float c;
  uint64_t seed;
  int64_t a_step, b_step;  // product blockIdx.y of a batch: elements between the operands; its C follows the others'
};

// Row tile bx and slice bz of nz of product by.
template <bool DROP>
__device__ __forceinline__ void skinny_nt_body(NtArgs p, int bx, int by, int bz, int nz) {
  p.A += by * p.a_step;
  p.B += by * p.b_step;
  p.C += (int64_t)by * nz * p.M * SJ;
  __shared__ __attribute__((aligned(1024))) uint16_t sA[kNtStages][SM * SK];
  __shared__ __attribute__((aligned(1024))) uint16_t sB[kNtStages][SJ * SK];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m0 = (int64_t)bx * SM;
  const int64_t kz0 = (int64_t)bz * p.k_split;
  const int64_t kz1 = (kz0 + p.k_split < p.K) ? kz0 + p.k_split : p.K;
  const int nk = kz0 < kz1 ? (int)((kz1 - kz0) / SK) : 0;

  // per-lane 32-bit offsets of the direct-to-LDS copies (8 rows x 128 B per instruction)
  const int lr = lane >> 3;
  uint32_t offA[4], offB[2];
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // A: 128 rows = 16 instructions, 4 per wave
    const int rloc = (wave * 4 + j) * 8 + lr;
    int64_t r = m0 + rloc;
    if (r > p.M - 1) r = p.M - 1;
    offA[j] = (uint32_t)((r * p.lda + (((lane & 7) ^ sk_swz(rloc)) * 8)) * 2);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {  // B: 64 rows = 8 instructions, 2 per wave
    const int rloc = (wave * 2 + j) * 8 + lr;
    offB[j] = (uint32_t)((rloc * p.ldb + (((lane & 7) ^ sk_swz(rloc)) * 8)) * 2);
  }
  // The copies are issued from inline assembly (uniform base in SGPRs, the
  // lane's offset in a VGPR): with the compiler builtin for them, the
  // generated code waited for every copy in flight, the next stages'
  // included, before the first LDS read of each stage, so no copy overlapped
  // the MFMAs. The explicit vmcnt before each stage's barrier is the only
  // wait on them.
  auto copy = [&](const char* base, uint32_t off, const uint16_t* lds) {
    const uint32_t m0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void_t*)lds);
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" :: "v"(off), "s"(base), "s"(m0)
                 : "memory", "m0");
  };
  auto issue = [&](int st, int buf) {
    const int64_t k0 = kz0 + (int64_t)st * SK;
    const char* a = reinterpret_cast<const char*>(p.A + k0);
    const char* b = reinterpret_cast<const char*>(p.B + k0);
#pragma unroll
    for (int j = 0; j < 4; ++j) copy(a, offA[j], sA[buf] + (wave * 4 + j) * 8 * SK);
#pragma unroll
    for (int j = 0; j < 2; ++j) copy(b, offB[j], sB[buf] + (wave * 2 + j) * 8 * SK);
  };

  f32x16_t acc[2];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[t][v] = 0.0f;

#pragma unroll
  for (int s = 0; s < kNtStages - 1; ++s)
    if (s < nk) issue(s, s);
  for (int st = 0; st < nk; ++st) {
    const int buf = st % kNtStages;
    if (st + 1 < nk) asm volatile("s_waitcnt vmcnt(6)" ::: "memory");  // stage st+1 (6 loads) may stay in flight
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (st + kNtStages - 1 < nk) issue(st + kNtStages - 1, (st + kNtStages - 1) % kNtStages);
#pragma unroll
    for (int kk = 0; kk < SK / 16; ++kk) {
      const int ch = 2 * kk + (lane >> 5);
      bf16x8_t a = *reinterpret_cast<const bf16x8_t*>(sA[buf] + sk_off(wave * 32 + (lane & 31), ch));
      if constexpr (DROP) {
        // element indices of the 8 values: row m of X (row length lda), columns k .. k+7
        const int64_t e0 = (m0 + wave * 32 + (lane & 31)) * p.lda + kz0 + (int64_t)st * SK + ch * 8;
        const u32x4_t u0 = philox_block(e0 >> 2, p.seed), u1 = philox_block((e0 >> 2) + 1, p.seed);
        const u32x4_t v = __builtin_bit_cast(u32x4_t, a);
        a = __builtin_bit_cast(bf16x8_t, u32x4_t{dropout_pair(v.x, u0.x, u0.y, p.thr, p.c),
                                                 dropout_pair(v.y, u0.z, u0.w, p.thr, p.c),
                                                 dropout_pair(v.z, u1.x, u1.y, p.thr, p.c),
                                                 dropout_pair(v.w, u1.z, u1.w, p.thr, p.c)});
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const bf16x8_t b = *reinterpret_cast<const bf16x8_t*>(sB[buf] + sk_off(t * 32 + (lane & 31), ch));
        acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc[t], 0, 0, 0);
      }
    }
  }
  // C[z][m][j]: lane l, register v -> row (v%4) + 4(l/32) + 8(v/4), column l%32
  float* Cz = p.C + (int64_t)bz * p.M * SJ;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int j = t * 32 + (lane & 31);
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int64_t m = m0 + wave * 32 + (v & 3) + 4 * (lane >> 5) + 8 * (v >> 2);
      if (m < p.M) Cz[m * SJ + j] = acc[t][v];
    }
  }
}

template <bool DROP>
__global__ __launch_bounds__(kSkThreads) void skinny_nt_kernel(NtArgs p) {
  skinny_nt_body<DROP>(p, (int)blockIdx.x, 0, (int)blockIdx.z, (int)gridDim.z);
}

// Where workgroups of a job in a launch of several begin, and its grid.
struct JobGrid {
  int first, x, y, z;
  int end() const { return first + x * y * z; }
};

__global__ __launch_bounds__(kSkThreads) void skinny_nt_jobs_kernel(NtArgs a, NtArgs b, JobGrid ga, JobGrid gb) {
  const bool second = (int)blockIdx.x >= gb.first;
  const NtArgs& p = second ? b : a;
  const JobGrid& g = second ? gb : ga;
  const int id = (int)blockIdx.x - g.first, xy = g.x * g.y;
  skinny_nt_body<false>(p, id % g.x, id / g.x % g.y, id / xy, g.z);
}

// ---- TN: both operands run the reduction down their rows ----------------------------

struct TnArgs {
  const uint16_t* L;  // [M][ldl]  large operand (X or dY)
  const uint16_t* S;  // [M][lds]  small operand (U or T), r columns valid
  float* C;           // [Z][W][SJ]
  int64_t ldl, lds, M, W, r, m_split;
  uint32_t thr;       // DROP: keep iff the element's Philox word >= thr; kept values scaled by c
  float c;
  uint64_t seed;
  int64_t l_step, s_step;  // product blockIdx.y of a batch, as in NtArgs (without DROP)
  const int8_t* L8;        // INT8: L's codes [M][W] (W % 64 == 0) and their scales [W / 64][m_pad], finite up to m_pad
  const float* scales;     // (M rounded up to 64)
  int64_t m_pad;
};

template <bool DROP>
__global__ __launch_bounds__(kSkThreads) void skinny_tn_kernel(TnArgs p) {
  __shared__ __attribute__((aligned(1024))) uint16_t sL[SM * SK];  // [c][m]
  __shared__ __attribute__((aligned(1024))) uint16_t sS[SJ * SK];  // [j][m]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t c0 = (int64_t)blockIdx.x * SM;
  const int64_t mz0 = (int64_t)blockIdx.z * p.m_split;
  const int64_t mz1 = (mz0 + p.m_split < p.M) ? mz0 + p.m_split : p.M;

  // staging roles: L tile = 64 rows x 128 columns -> thread: row pair rp, two 8-column chunks
  const int l_cq = tid & 7, l_rp = tid >> 3;              // 8 threads per row pair, 32 row pairs
  // S tile = 64 rows x 64 columns -> thread: row pair, one 8-column chunk (first 256 threads)
  const int s_cq = tid & 7, s_rp = tid >> 3;

  f32x16_t acc[2];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[t][v] = 0.0f;

  u32x4_t lv[2][2], sv[2];
  auto load = [&](int64_t ms) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t m = ms + 2 * l_rp + h;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int64_t c = c0 + (l_cq * 2 + q) * 8;
        lv[h][q] = (m < mz1 && c < p.W) ? *reinterpret_cast<const u32x4_t*>(p.L + m * p.ldl + c)
                                        : u32x4_t{0, 0, 0, 0};
      }
      const int64_t cs = s_cq * 8;
      sv[h] = (m < mz1 && cs < p.r) ? *reinterpret_cast<const u32x4_t*>(p.S + m * p.lds + cs) : u32x4_t{0, 0, 0, 0};
    }
  };
  // write (m, m+1) pairs of column c as one dword at [c][m]
  auto put_pairs = [&](uint16_t* T, int cbase, const u32x4_t& r0, const u32x4_t& r1, int mloc) {
    const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w};
    const uint32_t w1[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t a = (e & 1) ? (w0[e >> 1] >> 16) : (w0[e >> 1] & 0xFFFFu);
      const uint32_t b = (e & 1) ? (w1[e >> 1] >> 16) : (w1[e >> 1] & 0xFFFFu);
      const int row = cbase + e;
      *reinterpret_cast<uint32_t*>(T + sk_off(row, mloc >> 3) + (mloc & 7)) = a | (b << 16);
    }
  };

  // DROP: the staged rows of L (row-major [M][W], W % 64 == 0) after dropout;
  // out-of-range values were loaded as 0 and stay 0
  auto drop = [&](int64_t ms) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t m = ms + 2 * l_rp + h;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int64_t e0 = m * p.W + c0 + (l_cq * 2 + q) * 8;  // multiple of 8: two Philox blocks
        const u32x4_t u0 = philox_block(e0 >> 2, p.seed), u1 = philox_block((e0 >> 2) + 1, p.seed);
        u32x4_t& v = lv[h][q];
        v = u32x4_t{dropout_pair(v.x, u0.x, u0.y, p.thr, p.c), dropout_pair(v.y, u0.z, u0.w, p.thr, p.c),
                    dropout_pair(v.z, u1.x, u1.y, p.thr, p.c), dropout_pair(v.w, u1.z, u1.w, p.thr, p.c)};
      }
    }
  };

  if (mz0 < mz1) load(mz0);
  for (int64_t ms = mz0; ms < mz1; ms += SK) {
    __syncthreads();  // previous stage's fragment reads are done
    if constexpr (DROP) drop(ms);
    const int mloc = 2 * l_rp;
#pragma unroll
    for (int q = 0; q < 2; ++q) put_pairs(sL, (l_cq * 2 + q) * 8, lv[0][q], lv[1][q], mloc);
    put_pairs(sS, s_cq * 8, sv[0], sv[1], 2 * s_rp);
    __syncthreads();
    if (ms + SK < mz1) load(ms + SK);  // next stage's global loads overlap the MFMAs
#pragma unroll
    for (int kk = 0; kk < SK / 16; ++kk) {
      const int ch = 2 * kk + (lane >> 5);
      const bf16x8_t a = *reinterpret_cast<const bf16x8_t*>(sL + sk_off(wave * 32 + (lane & 31), ch));
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const bf16x8_t b = *reinterpret_cast<const bf16x8_t*>(sS + sk_off(t * 32 + (lane & 31), ch));
        acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc[t], 0, 0, 0);
      }
    }
  }
  float* Cz = p.C + (int64_t)blockIdx.z * p.W * SJ;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int j = t * 32 + (lane & 31);
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int64_t c = c0 + wave * 32 + (v & 3) + 4 * (lane >> 5) + 8 * (v >> 2);
      if (c < p.W) Cz[c * SJ + j] = acc[t][v];
    }
  }
}

// skinny_tn_dma_kernel: the product of skinny_tn_kernel without dropout, with both
// operands copied global -> LDS by global_load_lds_dwordx4 in their memory
// layout (rows of 128 L columns and of 64 S columns, m running down the rows)
// into a ring of kTnStages stages, so that the copies of two stages are in
// flight while a third is multiplied. The MFMA fragments (8 consecutive m of
// one column) are read with the transpose read ds_read_b64_tr_b16: in each
// group of 16 lanes, lane i receives element i % 4 of the 8 bytes that lane
// 4e + i / 4 addresses, as its element e. If lane j of the group addresses
// row m0 + j / 4, columns cb + 4 (j % 4) .. +3, lane i receives rows
// m0 .. m0 + 3 of column cb + i. Two such reads make one 8-element fragment.
// Rows outside the slice and S columns at or beyond r are copied from a
// zeroed 16-byte block, L columns at or beyond W from clamped (valid)
// addresses: their outputs are never stored. The results equal the
// register-staged kernel's bit for bit (the same MFMAs in the same order).
constexpr int kTnStages = 3;
constexpr int kTnLRow = SM * 2;                       // bytes per staged L row (128 columns)
constexpr int kTnSRow = SJ * 2;                       // bytes per staged S row (64 columns)
constexpr int kTnLBytes = SK * kTnLRow;               // 16 KB
constexpr int kTnStageBytes = kTnLBytes + SK * kTnSRow;  // 24 KB

__device__ __attribute__((aligned(16))) uint32_t g_tn_zero[4];  // zero-initialised copy source

// 16-byte chunk q of staged row m sits at chunk q ^ swz(m). L rows are 256 B
// (one row per pass of the 64 banks): the four rows that one transpose read
// of 32 lanes touches (m0 .. m0 + 3, four chunks each) land on 16 distinct
// chunk positions. S rows are 128 B (two rows per pass): rows m0 and m0 + 2
// are moved apart.
__device__ __forceinline__ int tn_lswz(int m) { return (m & 3) << 2; }
__device__ __forceinline__ int tn_sswz(int m) { return ((m >> 1) & 1) << 2; }

typedef short tn_v4i16 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ tn_v4i16 tn_read_tr(const char* lds_byte) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) tn_v4i16*)(lds_void_t*)lds_byte);
}

// INT8: the large operand as int8 values of blocks of 64 columns. Its codes lie in
// LDS as in memory (rows of 128 bytes); the transpose read of bytes
// (ds_read_b64_tr_b8: lane j of 16 addresses row j / 2, columns 8 (j % 2) .. +8, and
// receives column j of the 8 rows) gives a fragment's 8 codes of one column, which
// are multiplied with their rows' scales and rounded to bf16 in registers: the
// values of a dequantised copy, bit for bit, at half its bytes and without writing
// it: the linear's backward of 8192 rows, 4096 -> 11008, 809 -> 765 us; this launch
// 48-50 (the 11008 bf16 columns of dL2 in it), 4.4 TB/s.
typedef int tn_v2i32 __attribute__((ext_vector_type(2)));
constexpr int kTn8S = SK * SM, kTn8Scale = kTn8S + SK * kTnSRow;   // offsets of S and of the scales in a stage
static_assert(kTn8Scale + 1024 <= kTnStageBytes, "a stage of int8 values fits");
__device__ __forceinline__ int tn_8swz(int m) { return ((m >> 1) & 3) << 1; }   // of the 16-byte chunk of row m

// Column tile bx and slice bz of nz of product by.
template <bool INT8>
__device__ __forceinline__ void skinny_tn_body(TnArgs p, char* ring, int bx, int by, int bz, int nz) {
  p.L += by * p.l_step;
  p.S += by * p.s_step;
  p.C += (int64_t)by * nz * p.W * SJ;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t c0 = (int64_t)bx * SM;
  const int64_t mz0 = (int64_t)bz * p.m_split;
  const int64_t mz1 = (mz0 + p.m_split < p.M) ? mz0 + p.m_split : p.M;
  const int ns = mz0 < mz1 ? (int)((mz1 - mz0 + SK - 1) / SK) : 0;
  const char* zero = reinterpret_cast<const char*>(g_tn_zero);

  // Copy roles. L: instruction i of wave w moves rows 4 (4w + i) .. +3, lane
  // -> row 4 (4w + i) + lane / 16, chunk position lane % 16. S: instruction i
  // moves rows 8 (2w + i) .. +7, lane -> row 8 (2w + i) + lane / 8, position
  // lane % 8. The column parts of the source addresses are fixed per lane.
  // INT8: L instruction i moves rows 8 (2w + i) .. +7, lane -> row + lane / 8, chunk position lane % 8; every wave copies
  // the stage's scales too (the same bytes), 64 floats of both 64-column blocks.
  constexpr int kL = INT8 ? 2 : 4, kCopies = INT8 ? 5 : 6, kSAt = INT8 ? kTn8S : kTnLBytes;
  int64_t l_col[kL], s_col[2];
  bool s_in[2];
#pragma unroll
  for (int i = 0; i < kL; ++i) {
    if constexpr (INT8) {
      const int row = 8 * (2 * wave + i) + (lane >> 3);
      int64_t c = c0 + 16 * ((lane & 7) ^ tn_8swz(row));
      if (c > p.W - 16) c = p.W - 16;
      l_col[i] = c;
    } else {
      const int row = 4 * (4 * wave + i) + (lane >> 4);
      int64_t c = c0 + 8 * ((lane & 15) ^ tn_lswz(row));
      if (c > p.W - 8) c = p.W - 8;  // W % 8 == 0
      l_col[i] = c;
    }
  }
  const float* scale_at = nullptr;
  if constexpr (INT8) {
    int64_t blk = c0 / 64 + ((lane >> 4) & 1);
    if (blk > p.W / 64 - 1) blk = p.W / 64 - 1;
    scale_at = p.scales + blk * p.m_pad + 4 * (lane & 15);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = 8 * (2 * wave + i) + (lane >> 3);
    const int j = 8 * ((lane & 7) ^ tn_sswz(row));
    s_in[i] = j < p.r;
    s_col[i] = s_in[i] ? j : 0;
  }
  auto copy = [&](const char* src, char* lds) {
    const uint32_t m0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void_t*)lds);
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" :: "v"(src), "s"(m0) : "memory", "m0");
  };
  auto issue = [&](int st) {  // the kCopies copy instructions of this wave for stage st
    const int64_t ms = mz0 + (int64_t)st * SK;
    char* buf = ring + (st % kTnStages) * kTnStageBytes;
#pragma unroll
    for (int i = 0; i < kL; ++i) {
      const int row = INT8 ? 8 * (2 * wave + i) + (lane >> 3) : 4 * (4 * wave + i) + (lane >> 4);
      const int64_t m = ms + row;
      const char* from = INT8 ? reinterpret_cast<const char*>(p.L8 + m * p.W + l_col[i])
                              : reinterpret_cast<const char*>(p.L + m * p.ldl + l_col[i]);
      copy(m < mz1 ? from : zero, buf + (kL * wave + i) * 1024);
    }
    if constexpr (INT8) copy(reinterpret_cast<const char*>(scale_at + ms), buf + kTn8Scale);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = 8 * (2 * wave + i) + (lane >> 3);
      const int64_t m = ms + row;
      const char* src = (m < mz1 && s_in[i]) ? reinterpret_cast<const char*>(p.S + m * p.lds + s_col[i]) : zero;
      copy(src, buf + kSAt + (2 * wave + i) * 1024);
    }
  };

  f32x16_t acc[2];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[t][v] = 0.0f;

  // Transpose-read addresses, relative to a stage buffer and k-step: lane j
  // of its group addresses row (lane / 32) * 8 + 4 h + j / 4 (+16 kk),
  // columns cb + 4 (j % 4) .. +3 with cb = 16 ((lane / 16) % 2) + the wave's
  // (L) or the tile's (S) first column.
  const int jl = lane & 15;
  const int rbase = 8 * (lane >> 5) + (jl >> 2);
  const int cl = wave * 32 + 16 * ((lane >> 4) & 1) + 4 * (jl & 3);  // L column (within the tile)
  const int cs = 16 * ((lane >> 4) & 1) + 4 * (jl & 3);              // S column within a 32-wide tile
  auto loff = [&](int row) { return row * kTnLRow + ((((cl >> 3) ^ tn_lswz(row))) << 4) + ((cl & 7) << 1); };
  auto soff = [&](int row, int t) {
    const int c = 32 * t + cs;
    return kSAt + row * kTnSRow + (((c >> 3) ^ tn_sswz(row)) << 4) + ((c & 7) << 1);
  };

#pragma unroll
  for (int st = 0; st < kTnStages - 1; ++st)
    if (st < ns) issue(st);
  for (int st = 0; st < ns; ++st) {
    // this wave's copies of stage st are complete (those of st + 1 may not be)
    if (st + 1 < ns) asm volatile("s_waitcnt vmcnt(%0)" :: "n"(kCopies) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();  // every wave's copies of stage st are visible; stage st-1's reads are done
    if (st + kTnStages - 1 < ns) issue(st + kTnStages - 1);  // into stage st-1's buffer
    const char* buf = ring + (st % kTnStages) * kTnStageBytes;
#pragma unroll
    for (int kk = 0; kk < SK / 16; ++kk) {
      const int r0 = 16 * kk + rbase;
      bf16x8_t a;
      if constexpr (INT8) {
        const int m = 16 * kk + 8 * (lane >> 5), row = m + (jl >> 1);
        const int c = 2 * wave + ((lane >> 4) & 1);
        const char* at = buf + row * SM + ((c ^ tn_8swz(row)) << 4) + 8 * (jl & 1);
        const tn_v2i32 q = __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) tn_v2i32*)(lds_void_t*)at);
        const f32x4_t* sc = reinterpret_cast<const f32x4_t*>(buf + kTn8Scale + 256 * (wave >> 1) + 4 * m);
        const f32x4_t s0 = sc[0], s1 = sc[1];
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = (float)(int8_t)(q.x >> (8 * e)) * s0[e];
          x[4 + e] = (float)(int8_t)(q.y >> (8 * e)) * s1[e];
        }
        a = __builtin_bit_cast(bf16x8_t, u32x4_t{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                                 pack_bf16x2(x[6], x[7])});
      } else {
        const tn_v4i16 a0 = tn_read_tr(buf + loff(r0)), a1 = tn_read_tr(buf + loff(r0 + 4));
        a = __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7));
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const tn_v4i16 b0 = tn_read_tr(buf + soff(r0, t)), b1 = tn_read_tr(buf + soff(r0 + 4, t));
        const bf16x8_t b = __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7));
        acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc[t], 0, 0, 0);
      }
    }
  }
  float* Cz = p.C + (int64_t)bz * p.W * SJ;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int j = t * 32 + (lane & 31);
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int64_t c = c0 + wave * 32 + (v & 3) + 4 * (lane >> 5) + 8 * (v >> 2);
      if (c < p.W) Cz[c * SJ + j] = acc[t][v];
    }
  }
}

__global__ __launch_bounds__(kSkThreads) void skinny_tn_dma_kernel(TnArgs p) {
  __shared__ __attribute__((aligned(1024))) char ring[kTnStages * kTnStageBytes];
  skinny_tn_body<false>(p, ring, (int)blockIdx.x, 0, (int)blockIdx.z, (int)gridDim.z);
}

// FIRST8: the first job's large operand is int8 values.
template <bool FIRST8>
__global__ __launch_bounds__(kSkThreads) void skinny_tn_jobs_kernel(TnArgs a, TnArgs b, JobGrid ga, JobGrid gb) {
  const bool second = (int)blockIdx.x >= gb.first;
  const TnArgs& p = second ? b : a;
  const JobGrid& g = second ? gb : ga;
  const int id = (int)blockIdx.x - g.first, xy = g.x * g.y;
  __shared__ __attribute__((aligned(1024))) char ring[kTnStages * kTnStageBytes];
  if (FIRST8 && !second) skinny_tn_body<true>(a, ring, id % g.x, id / g.x % g.y, id / xy, g.z);
  else skinny_tn_body<false>(p, ring, id % g.x, id / g.x % g.y, id / xy, g.z);
}

// sum_z P[z slab .. +4], in order, 8 slices' loads in flight (one at a time, the
// sum of 32 slices of 391 rows took 10 us).
__device__ __forceinline__ f32x4_t sum_slices(const float* __restrict__ P, int Z, int64_t slab) {
  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  int z = 0;
  for (; z + 8 <= Z; z += 8) {
    f32x4_t v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = *reinterpret_cast<const f32x4_t*>(P + (int64_t)(z + u) * slab);
#pragma unroll
    for (int u = 0; u < 8; ++u) acc += v[u];
  }
  for (; z < Z; ++z) acc += *reinterpret_cast<const f32x4_t*>(P + (int64_t)z * slab);
  return acc;
}

// out = alpha * sum_z P[z] over a [rows][SJ] slab, columns j < r:
//   mode 0: out[m][j] (columns [r, ldo) zero) in bf16, plus
//           optional out2[m][j] = bf16(alpha2 * sum) with row stride r
//   mode 1: out[m][j] fp32 or bf16
// out's rows are `pitch` elements apart.
// Four consecutive columns per thread (r % 8 == 0 and ldo % 4 == 0, so a
// group of four is all below r or all at or above it): 16-byte partial loads,
// the sum over z in order, 8- or 16-byte stores.
struct ReduceArgs {
  const float* P;
  int Z;
  int64_t rows;
  int r;
  float alpha;
  int mode, out_bf16;
  void* out;
  int64_t ldo;
  float alpha2;
  uint16_t* out2;
  int64_t pitch;
  int64_t o_step, o2_step;   // elements between the results of a batch
};

// Workgroup bx of nx of product by.
__device__ __forceinline__ void skinny_reduce_body(const ReduceArgs& a, int bx, int nx, int by) {
  const int r = a.r;
  const float* P = a.P + (int64_t)by * a.Z * a.rows * SJ;
  void* out = a.out_bf16 ? (void*)(static_cast<uint16_t*>(a.out) + by * a.o_step) : (void*)(static_cast<float*>(a.out) + by * a.o_step);
  uint16_t* out2 = a.out2 ? a.out2 + by * a.o2_step : nullptr;
  const int64_t width = (a.mode == 0) ? a.ldo : r;
  const int64_t w4 = width / 4;
  const int64_t total = a.rows * w4;
  const int64_t slab = a.rows * SJ;
  for (int64_t i = (int64_t)bx * 256 + threadIdx.x; i < total; i += (int64_t)nx * 256) {
    const int64_t m = i / w4, j = (i - m * w4) * 4;
    const int64_t o = m * a.pitch + j;
    if (j >= r) {
      *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(out) + o) = u32x2_t{0u, 0u};
      continue;
    }
    const f32x4_t acc = sum_slices(P + m * SJ + j, a.Z, slab);
    const f32x4_t v = {a.alpha * acc.x, a.alpha * acc.y, a.alpha * acc.z, a.alpha * acc.w};
    if (a.out_bf16)
      *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(out) + o) = u32x2_t{pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
    else
      *reinterpret_cast<f32x4_t*>(static_cast<float*>(out) + o) = v;
    if (a.mode == 0 && out2)
      *reinterpret_cast<u32x2_t*>(out2 + m * r + j) =
          u32x2_t{pack_bf16x2(a.alpha2 * acc.x, a.alpha2 * acc.y), pack_bf16x2(a.alpha2 * acc.z, a.alpha2 * acc.w)};
  }
}

__global__ __launch_bounds__(256) void skinny_reduce_kernel(ReduceArgs a) {
  skinny_reduce_body(a, (int)blockIdx.x, (int)gridDim.x, 0);
}

// Transposed reduction: out[j][c] = alpha * sum_z P[z][c][j] for j < r, c < W,
// output row stride W. One workgroup per 64 columns c and 16 ranks j (so
// that even W = 4096 gives 256 workgroups): each thread sums 4 ranks of one
// column over the Z partial tiles in a fixed z order (16-byte loads), the
// 64 x 16 result is transposed through LDS, and each output row segment is
// written 4 columns per thread.
// (ReduceArgs: rows is W.) Columns 64 bx .. of rank block by of product bz.
__device__ __forceinline__ void skinny_reduce_t_body(const ReduceArgs& a, int bx, int by, int bz) {
  __shared__ float tile[64][16 + 1];
  const int64_t W = a.rows;
  const int r = a.r;
  const float* P = a.P + (int64_t)bz * a.Z * W * SJ;
  void* out = a.out_bf16 ? (void*)(static_cast<uint16_t*>(a.out) + bz * a.o_step) : (void*)(static_cast<float*>(a.out) + bz * a.o_step);
  const int t = threadIdx.x;
  const int64_t c0 = (int64_t)bx * 64;
  const int j0 = by * 16;
  if (j0 >= r) return;                         // uniform per workgroup
  const int cl = t >> 2, jq = (t & 3) * 4;     // column c0 + cl, ranks j0 + jq .. +4
  const int64_t c = c0 + cl;
  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < W) acc = sum_slices(P + c * SJ + j0 + jq, a.Z, W * SJ);
#pragma unroll
  for (int e = 0; e < 4; ++e) tile[cl][jq + e] = acc[e];
  __syncthreads();
  const int jl = t >> 4, cq = (t & 15) * 4;   // rank j0 + jl, columns c0 + cq .. +4
  const int j = j0 + jl;
  if (j < r) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t cc = c0 + cq + e;
      if (cc < W) {
        const float v = a.alpha * tile[cq + e][jl];
        if (a.out_bf16) static_cast<uint16_t*>(out)[(int64_t)j * W + cc] = f32_to_bf16(v);
        else static_cast<float*>(out)[(int64_t)j * W + cc] = v;
      }
    }
  }
}

__global__ __launch_bounds__(256) void skinny_reduce_t_kernel(ReduceArgs a) {
  skinny_reduce_t_body(a, (int)blockIdx.x, (int)blockIdx.y, 0);
}

// The sums of two jobs and of a product cut into slices (values 0: none), in one launch.
struct SumJob {
  ReduceArgs a;
  int transpose;
  JobGrid g;
};

__global__ __launch_bounds__(256) void skinny_sums_kernel(SumJob p, SumJob q, SplitSum s, int first_split) {
  const int id = (int)blockIdx.x;
  if (id >= first_split) {
    split_sum_body(s, (int64_t)(id - first_split) * 256 + threadIdx.x);
    return;
  }
  const SumJob& j = id >= q.g.first ? q : p;
  const int i = id - j.g.first;
  if (j.transpose) skinny_reduce_t_body(j.a, i % j.g.x, i / j.g.x % j.g.y, i / (j.g.x * j.g.y));
  else skinny_reduce_body(j.a, i % j.g.x, j.g.x, i / j.g.x);
}

int64_t sk_cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

int64_t sk_grid(int64_t total) {
  int64_t b = sk_cdiv(total, 256);
  if (b > 8192) b = 8192;
  return b < 1 ? 1 : b;
}

}  // namespace

// Number of reduction slices for a skinny product with `tiles` output tiles
// over a reduction of length klen (multiples of 64): about 512 workgroups
// stream the large operand, or, with fit > 0, at most max(fit, tiles) of
// them (the workgroups that fit on the device at once), so that none waits
// for a second round.
SkinnySplit skinny_split(int64_t tiles, int64_t klen, int64_t fit) {
  const int64_t steps = sk_cdiv(klen, SK);
  if (steps < 1) return SkinnySplit{1, SK};
  int64_t z = fit > 0 ? fit / (tiles < 1 ? 1 : tiles) : sk_cdiv(512, tiles < 1 ? 1 : tiles);
  if (z > 32) z = 32;
  if (z > steps) z = steps;
  if (z < 1) z = 1;
  const int64_t per = sk_cdiv(steps, z);
  SkinnySplit s;
  s.len = per * SK;
  s.Z = (int)sk_cdiv(steps, per);
  if (s.Z < 1) s.Z = 1;
  return s;
}

size_t skinny_partial_bytes(int64_t M, int64_t K, int64_t N) {
  const SkinnySplit a = skinny_split(sk_cdiv(M, SM), K);
  const SkinnySplit b = skinny_split(sk_cdiv(M, SM), N);
  const SkinnySplit c = skinny_split(sk_cdiv(K, SM), M);
  const SkinnySplit d = skinny_split(sk_cdiv(N, SM), M);
  size_t m = (size_t)a.Z * M;
  if ((size_t)b.Z * M > m) m = (size_t)b.Z * M;
  if ((size_t)c.Z * K > m) m = (size_t)c.Z * K;
  if ((size_t)d.Z * N > m) m = (size_t)d.Z * N;
  return m * SJ * sizeof(float);
}

size_t skinny_partial_bound(int64_t M, int64_t K, int64_t N) {
  const int64_t fit = 2 * (int64_t)device_cu_count() > 512 ? 2 * (int64_t)device_cu_count() : 512;
  auto least = [](int64_t x, int64_t y) { return x < y ? x : y; };
  const int64_t steps = sk_cdiv(K > N ? K : N, SK);
  int64_t rows = least(least(32, steps) * M, fit * SM + M);   // slices x rows: at most fit / (M / SM) + 1 slices
  for (const int64_t W : {K, N}) {
    const int64_t z = least(least(32, sk_cdiv(fit, sk_cdiv(W, SM))), sk_cdiv(M, SK));
    if (z * W > rows) rows = z * W;
  }
  return (size_t)rows * SJ * sizeof(float);
}

namespace {

NtArgs nt_args(const SkinnyNt& j, const SkinnySplit& sp, float* part) {
  NtArgs a{};
  a.A = j.A; a.B = j.B; a.C = part; a.lda = j.lda; a.ldb = j.ldb; a.M = j.M; a.K = j.K; a.k_split = sp.len;
  a.c = 1.0f;
  a.a_step = j.batch.a_step; a.b_step = j.batch.b_step;
  return a;
}

SkinnySplit nt_split(const SkinnyNt& j) {
  // 72 KB of LDS: two workgroups per CU
  return skinny_split(sk_cdiv(j.M, SM), j.K, 2 * (int64_t)device_cu_count());
}

ReduceArgs nt_reduce(const SkinnyNt& j, const SkinnySplit& sp, const float* part) {
  return ReduceArgs{part, sp.Z, j.M, j.r, j.alpha, 0, 1, j.out, j.ldo, j.alpha2, j.out2, j.pitch ? j.pitch : j.ldo,
                    j.batch.o_step, j.batch.o2_step};
}

TnArgs tn_args(const SkinnyTn& j, const SkinnySplit& sp, float* part) {
  TnArgs a{};
  a.L = j.L; a.S = j.S; a.C = part; a.ldl = j.ldl; a.lds = j.lds; a.M = j.M; a.W = j.W; a.r = j.r; a.m_split = sp.len;
  a.c = 1.0f;
  a.l_step = j.batch.a_step; a.s_step = j.batch.b_step;
  a.L8 = j.L8; a.scales = j.scales; a.m_pad = sk_cdiv(j.M, SK) * SK;
  return a;
}

SkinnySplit tn_split(const SkinnyTn& j) {
  // the copy-ring kernel (72 KB of LDS) fits two workgroups per CU
  return skinny_split(sk_cdiv(j.W, SM), j.M, 2 * (int64_t)device_cu_count());
}

ReduceArgs tn_reduce(const SkinnyTn& j, const SkinnySplit& sp, const float* part) {
  return ReduceArgs{part, sp.Z, j.W, j.r, j.alpha, 1, j.out_bf16 ? 1 : 0, j.out, (int64_t)j.r, 0.0f, nullptr, (int64_t)j.r,
                    j.batch.o_step, 0};
}

SumJob sum_job(const ReduceArgs& a, bool transpose, int n, int first) {
  SumJob s{a, transpose ? 1 : 0, JobGrid{first, 0, 1, n}};
  if (transpose) {
    s.g.x = (int)sk_cdiv(a.rows, 64);
    s.g.y = (a.r + 15) / 16;
  } else {
    s.g.x = (int)sk_grid(a.rows * (a.mode == 0 ? a.ldo : a.r) / 4);
    if (s.g.x > 1024) s.g.x = 1024;
  }
  return s;
}

hipError_t launch_sums(const SumJob& p, const SumJob& q, const SplitSum* split, hipStream_t stream) {
  const int first = q.g.end();
  const SplitSum s = split ? *split : SplitSum{nullptr, nullptr, 0, 0};
  const int64_t blocks = first + (s.values / 8 + 255) / 256;
  hipLaunchKernelGGL(skinny_sums_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, p, q, s, first);
  return hipGetLastError();
}

}  // namespace

hipError_t skinny_nt_jobs(const SkinnyNt* jobs, int n, float* part, hipStream_t stream) {
  const SkinnyNt& ja = jobs[0];
  const SkinnySplit sa = nt_split(ja);
  const JobGrid ga{0, (int)sk_cdiv(ja.M, SM), ja.batch.n, sa.Z};
  const NtArgs a = nt_args(ja, sa, part);
  NtArgs b = a;
  JobGrid gb{ga.end(), 1, 1, 0};                // no second job: no workgroups
  SumJob p = sum_job(nt_reduce(ja, sa, part), false, ja.batch.n, 0), q = p;
  q.g = JobGrid{p.g.end(), 1, 1, 0};
  if (n > 1) {
    const SkinnyNt& jb = jobs[1];
    const SkinnySplit sb = nt_split(jb);
    float* more = part + (int64_t)ja.batch.n * sa.Z * ja.M * SJ;
    gb = JobGrid{ga.end(), (int)sk_cdiv(jb.M, SM), jb.batch.n, sb.Z};
    b = nt_args(jb, sb, more);
    q = sum_job(nt_reduce(jb, sb, more), false, jb.batch.n, p.g.end());
  }
  hipLaunchKernelGGL(skinny_nt_jobs_kernel, dim3((unsigned)gb.end()), dim3(kSkThreads), 0, stream, a, b, ga, gb);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_sums(p, q, nullptr, stream);
}

hipError_t skinny_tn_jobs(const SkinnyTn* jobs, int n, float* part, const SplitSum* split, hipStream_t stream) {
  const SkinnyTn& ja = jobs[0];
  const SkinnySplit sa = tn_split(ja);
  const JobGrid ga{0, (int)sk_cdiv(ja.W, SM), ja.batch.n, sa.Z};
  const TnArgs a = tn_args(ja, sa, part);
  TnArgs b = a;
  JobGrid gb{ga.end(), 1, 1, 0};
  SumJob p = sum_job(tn_reduce(ja, sa, part), ja.transpose, ja.batch.n, 0), q = p;
  q.g = JobGrid{p.g.end(), 1, 1, 0};
  if (n > 1) {
    const SkinnyTn& jb = jobs[1];
    const SkinnySplit sb = tn_split(jb);
    float* more = part + (int64_t)ja.batch.n * sa.Z * ja.W * SJ;
    gb = JobGrid{ga.end(), (int)sk_cdiv(jb.W, SM), jb.batch.n, sb.Z};
    b = tn_args(jb, sb, more);
    q = sum_job(tn_reduce(jb, sb, more), jb.transpose, jb.batch.n, p.g.end());
  }
  if (ja.L8)
    hipLaunchKernelGGL(skinny_tn_jobs_kernel<true>, dim3((unsigned)gb.end()), dim3(kSkThreads), 0, stream, a, b, ga, gb);
  else
    hipLaunchKernelGGL(skinny_tn_jobs_kernel<false>, dim3((unsigned)gb.end()), dim3(kSkThreads), 0, stream, a, b, ga, gb);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_sums(p, q, split, stream);
}

// C = A B^T over K with B [64][ldb] (rows >= r zero), then reduce.
hipError_t skinny_nt(const uint16_t* A, int64_t lda, const uint16_t* B, int64_t ldb, int64_t M, int64_t K, int r,
                     float* part, float alpha, uint16_t* out, int64_t ldo, float alpha2, uint16_t* out2,
                     hipStream_t stream, const DropoutParams* dr) {
  if (dr && lda != K) return hipErrorInvalidValue;  // the mask indexes a contiguous [M][K] input
  const SkinnyNt j{A, lda, B, ldb, M, K, r, alpha, out, ldo, 0, alpha2, out2, SkinnyBatch{1, 0, 0, 0, 0}};
  const SkinnySplit sp = nt_split(j);
  NtArgs a = nt_args(j, sp, part);
  if (dr) {
    a.thr = dr->thr; a.c = dr->c; a.seed = dr->seed;
  }
  const dim3 grid((unsigned)sk_cdiv(M, SM), 1, (unsigned)sp.Z);
  if (dr)
    hipLaunchKernelGGL(skinny_nt_kernel<true>, grid, dim3(kSkThreads), 0, stream, a);
  else
    hipLaunchKernelGGL(skinny_nt_kernel<false>, grid, dim3(kSkThreads), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(skinny_reduce_kernel, dim3((unsigned)sk_grid(M * ldo / 4)), dim3(256), 0, stream, nt_reduce(j, sp, part));
  return hipGetLastError();
}

// C[c][j] = sum_m L[m][c] S[m][j], then reduce to out (transposed if `transpose`).
hipError_t skinny_tn(const uint16_t* L, int64_t ldl, int64_t W, const uint16_t* S, int64_t lds, int64_t M, int r,
                     float* part, float alpha, bool transpose, bool out_bf16, void* out, hipStream_t stream,
                     const DropoutParams* dr) {
  if (dr && (ldl != W || W % 64)) return hipErrorInvalidValue;  // the mask indexes a contiguous [M][W] input
  const SkinnyTn j{L, ldl, W, S, lds, M, r, alpha, transpose, out_bf16, out, SkinnyBatch{1, 0, 0, 0, 0}, nullptr, nullptr};
  const SkinnySplit sp = dr ? skinny_split(sk_cdiv(W, SM), M, 0) : tn_split(j);
  TnArgs a = tn_args(j, sp, part);
  if (dr) {
    a.thr = dr->thr; a.c = dr->c; a.seed = dr->seed;
  }
  const dim3 grid((unsigned)sk_cdiv(W, SM), 1, (unsigned)sp.Z);
  if (dr)
    hipLaunchKernelGGL(skinny_tn_kernel<true>, grid, dim3(kSkThreads), 0, stream, a);
  else
    hipLaunchKernelGGL(skinny_tn_dma_kernel, grid, dim3(kSkThreads), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const ReduceArgs ra = tn_reduce(j, sp, part);
  if (transpose)
    hipLaunchKernelGGL(skinny_reduce_t_kernel, dim3((unsigned)sk_cdiv(W, 64), SJ / 16), dim3(256), 0, stream, ra);
  else
    hipLaunchKernelGGL(skinny_reduce_kernel, dim3((unsigned)sk_grid(W * (int64_t)r / 4)), dim3(256), 0, stream, ra);
  return hipGetLastError();
}

}  // namespace qlora
