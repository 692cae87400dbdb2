// Core of the bf16 MFMA products with an epilogue of their own (gated.hip,
// head.hip), for gfx950: one workgroup of 8 waves computes a TM x 256 tile of
//
//   C[m][n] = sum_k A[m][k] B[n][k]  (+ sum_j A2[m][j] B2[n][j])
//
// in fp32 accumulators and hands them to the caller's epilogue. Each operand is
// either row-major (the reduction contiguous in a row) or k-major (the reduction
// down the rows: B stored [k][n]); a k-major tile lies in LDS as it lies in
// memory, and its fragments are read with the LDS transpose read.
//
// Schedule (that of the dense linear's GEMM): stages of 64 k, copied global ->
// LDS without registers, A double- and B triple-buffered (160 KB); fragments of
// k-step kk + 1 are read while the MFMAs of kk run; the copies of stage st + 2
// go out one instruction at a time among the MFMAs of stage st. A wave owns
// TM / 2 x 64 outputs as 32 x 32 x 16 MFMA accumulators. Large products: 8192 x
// 4096 x 22016 with B k-major 1.35 PFLOP/s, 6144 x 32000 x 4096 with both row-major
// and P's epilogue 1.18-1.25 (a large library product 1.46).
//
// Copies take a uniform 64-bit base per tile and stage and a 32-bit offset per
// lane (inside the tile; k-major: inside 96 rows, so rows of up to 2^24 elements),
// so operands of any number of rows can be read. Rows past the end of
// an operand are read from its last row: what they give is never stored, or, down
// a reduction, meets zeros of the other operand.
#pragma once

#include "common.h"
#include "launch.h"

#include <type_traits>

namespace qlora {

typedef __attribute__((address_space(3))) void tg_lds_t;
typedef short tg_v4i16 __attribute__((ext_vector_type(4)));

constexpr int kTgN = 256, kTgK = 64, kTgWaves = 8, kTgThreads = 64 * kTgWaves;
constexpr int kTgStage = 256 * kTgK;               // LDS elements per operand and stage
constexpr int kTgSmem = 5 * kTgStage;              // A x 2, B x 3

struct TgOperand {
  const uint16_t* p;
  int64_t ld;      // elements between rows
  int64_t n;       // row-major: rows; k-major: columns (a multiple of 8)
};

struct TgArgs {
  TgOperand A, B, A2, B2;
  int64_t kmain, kslab;        // reductions, multiples of 64 (kslab 0: none)
  int64_t krows_a, krows_b;    // k-major operands: rows that exist (the last one stands for those past it)
  int per_slice;               // stages per reduction slice
};

// The operands' layouts and what a stage means.
//   AK, BK  the operand is k-major
//   SLAB    there is a second pair of operands, in the same layouts
//   PAIRED  B (k-major, main) has its rows in pairs of blocks: block b of 32 rows
//           of the first half at 64 b, of the second half at 64 b + 32
template <bool AK, bool BK, bool SLAB, bool PAIRED>
struct TgLayout {
  static constexpr bool kAK = AK, kBK = BK, kSlab = SLAB, kPaired = PAIRED;
};

__device__ __forceinline__ int tg_swz(int row) { return (row >> 1) & 7; }     // row-major stage rows (128 bytes)

// One stage of an operand, W rows (row-major) or columns (k-major) wide: this
// wave's copy instruction j of NI. Lane i of an instruction writes 16 bytes at
// 16 i of a 1 KB slice.
//   row-major: 8 rows of 128 bytes; chunk c of row r at c ^ tg_swz(r)
//   k-major: 512 / W rows of 2 W bytes; chunk c of row k at c ^ 4 (k % 4): the
//   four rows that a transpose read touches lie in different banks
__device__ __forceinline__ void tg_copy(const char* base, uint32_t off, uint16_t* lds, int slice) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(tg_lds_t*)(lds + slice * 512));
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" :: "v"(off), "s"(base), "s"(m0)
               : "memory", "m0");
}

// The lane's place in copy instruction j: its row in the stage (row-major: tile row, k-major: k) and 16-byte chunk.
template <int W, bool KMAJOR, int NI>
__device__ __forceinline__ void tg_place(int j, int* row, int* chunk) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slice = wave * NI + j;
  if constexpr (KMAJOR) {
    constexpr int kLanes = W / 8;                     // per k row
    *row = slice * (64 / kLanes) + lane / kLanes;
    *chunk = (lane % kLanes) ^ ((*row & 3) << 2);
  } else {
    *row = slice * 8 + (lane >> 3);
    *chunk = (lane & 7) ^ tg_swz(*row);
  }
}

// One operand's copies of a tile: the lane's byte offsets.
//   row-major: off, from the tile's first row (main and slab operands apart: their ld differ)
//   k-major: row, of the lane's k row in a stage, and off, of its columns from column 0; main and slab operands have
//   one ld and one width
template <int W, bool KMAJOR>
struct TgSource {
  static constexpr int kNi = W / 8 / kTgWaves;        // copy instructions per wave and stage
  uint32_t off[kNi], row[KMAJOR ? kNi : 1];
  __device__ __forceinline__ void init(const TgOperand& o, int64_t first) {
#pragma unroll
    for (int j = 0; j < kNi; ++j) {
      int r, chunk;
      tg_place<W, KMAJOR, kNi>(j, &r, &chunk);
      if constexpr (KMAJOR) {
        int64_t col = first + chunk * 8;
        if (col > o.n - 8) col = o.n - 8;
        off[j] = (uint32_t)(col * 2);
        row[j] = (uint32_t)(r * o.ld * 2);
      } else {
        const int64_t in = first + r < o.n ? r : o.n - 1 - first;
        off[j] = (uint32_t)((in * o.ld + chunk * 8) * 2);
      }
    }
  }
};

// The byte offset of the last k row that a stage at k0 may read, or of its row 63.
__device__ __forceinline__ uint32_t tg_limit(int64_t krows, int64_t k0, int64_t ld) {
  const int64_t last = krows - 1 - k0;
  return (uint32_t)((last < kTgK - 1 ? last : kTgK - 1) * ld * 2);
}

// Epilogue: a struct E with
//   template <int MI> __device__ void operator()(f32x16_t (&acc)[MI][2], int64_t m0, int64_t n0, int wm, int wn,
//                                                int z, uint16_t* smem) const;
// called by all waves after a barrier; register v of lane l of acc[i][j] is row
// m0 + wm 32 MI + 32 i + (v % 4) + 4 (l / 32) + 8 (v / 4), column n0 + 64 wn + 32 j + l % 32.
template <int TM, class L, class E>
__device__ __forceinline__ void tg_tile(const TgArgs& p, const E& epi, int64_t m0, int64_t n0, uint16_t* smem, int z) {
  constexpr int MI = TM / 64, NJ = 2;
  using SA = TgSource<TM, L::kAK>;
  using SB = TgSource<kTgN, L::kBK>;
  constexpr int NA = SA::kNi, NB = SB::kNi;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int nmain = (int)(p.kmain / kTgK);
  const int nall = nmain + (L::kSlab ? (int)(p.kslab / kTgK) : 0);
  const int s0 = z * p.per_slice;
  const int nk = (s0 + p.per_slice < nall ? s0 + p.per_slice : nall) - s0;   // stages of this slice (may be 0)

  f32x16_t acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  SA a1, a2;
  SB b1, b2;
  a1.init(p.A, m0);
  b1.init(p.B, n0);
  if constexpr (L::kSlab && !L::kAK) a2.init(p.A2, m0);
  if constexpr (L::kSlab && !L::kBK) b2.init(p.B2, n0);
  // PAIRED: k row 32 .. 63 of a main stage lies 32 rows further
  uint32_t pair[L::kPaired ? NB : 1];
  if constexpr (L::kPaired) {
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      int r, chunk;
      tg_place<kTgN, true, NB>(j, &r, &chunk);
      pair[j] = b1.row[j] + (uint32_t)((r & 32) * p.B.ld * 2);
    }
  }
  const char* const A1 = reinterpret_cast<const char*>(p.A.p + (L::kAK ? 0 : m0 * p.A.ld));
  const char* const B1 = reinterpret_cast<const char*>(p.B.p + (L::kBK ? 0 : n0 * p.B.ld));
  const char* const A2 = L::kSlab ? reinterpret_cast<const char*>(p.A2.p + (L::kAK ? 0 : m0 * p.A2.ld)) : nullptr;
  const char* const B2 = L::kSlab ? reinterpret_cast<const char*>(p.B2.p + (L::kBK ? 0 : n0 * p.B2.ld)) : nullptr;

  auto a_buf = [&](int st) { return smem + (st & 1) * kTgStage; };
  auto b_buf = [&](int st) { return smem + (2 + st % 3) * kTgStage; };
  // copy instruction q of stage st of the slice: q < NA are the A tile's, the rest the B tile's. Main and slab stages'
  // copies run in loops of their own: selected in one loop, they cut it into branches between the MFMAs.
  auto issue_one = [&](int st, int q, auto of_slab) {
    constexpr bool slab = L::kSlab && decltype(of_slab)::value;
    const int at = s0 + st;
    const int64_t k0 = (int64_t)(slab ? at - nmain : at) * kTgK;
    if (q < NA) {
      const char* base = slab ? A2 : A1;
      uint32_t off;
      if constexpr (L::kAK) {
        const uint32_t most = tg_limit(p.krows_a, k0, p.A.ld);
        off = a1.off[q] + (slab || a1.row[q] < most ? a1.row[q] : most);
        base += k0 * p.A.ld * 2;
      } else {
        off = slab ? a2.off[q] : a1.off[q];
        base += k0 * 2;
      }
      tg_copy(base, off, a_buf(st), wave * NA + q);
    } else {
      const int j = q - NA;
      const char* base = slab ? B2 : B1;
      uint32_t off;
      if constexpr (L::kBK) {
        int64_t first = k0;
        if constexpr (L::kPaired) {
          const bool second = at >= (int)(p.kmain / 2 / kTgK);
          if (!slab) first = 2 * (k0 - (second ? p.kmain / 2 : 0)) + (second ? 32 : 0);
          off = b1.off[j] + (slab ? b1.row[j] : pair[j]);
        } else {
          const uint32_t most = tg_limit(p.krows_b, k0, p.B.ld);
          off = b1.off[j] + (slab || b1.row[j] < most ? b1.row[j] : most);
        }
        base += first * p.B.ld * 2;
      } else {
        off = slab ? b2.off[j] : b1.off[j];
        base += k0 * 2;
      }
      tg_copy(base, off, b_buf(st), wave * NB + j);
    }
  };
  bf16x8_t fa[2][MI], fb[2][NJ];                      // two register sets of k-step fragments
  // k-major fragments: two transpose reads of 4 k each. Lane j of a group of 16 addresses row 16 kk + 8 (lane / 32)
  // + 4 h + j / 4, columns c + 4 (j % 4) .. +4, and receives column c + j of the four rows.
  const int jl = lane & 15, krow = 8 * (lane >> 5) + (jl >> 2), kcol = 16 * ((lane >> 4) & 1) + 4 * (jl & 3);
  const int kx = (jl >> 2) << 2;                      // chunk swizzle of the lane's rows
  auto frag_k = [&](const uint16_t* buf, int w, int col, int kk) {
    const int c = col + kcol;
    const char* at = reinterpret_cast<const char*>(buf) + (((c >> 3) ^ kx) << 4) + ((c & 7) << 1) + (krow + 16 * kk) * (2 * w);
    const tg_v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) tg_v4i16*)(tg_lds_t*)at);
    const tg_v4i16 hi =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) tg_v4i16*)(tg_lds_t*)(at + 8 * w));
    return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto frag_r = [&](const uint16_t* buf, int row, int kk) {
    const int ch = 2 * kk + (lane >> 5);
    row += lane & 31;
    return *reinterpret_cast<const bf16x8_t*>(buf + row * kTgK + ((ch ^ tg_swz(row)) << 3));
  };
  auto frag = [&](int st, int kk, int set) {
    const uint16_t* As = a_buf(st);
    const uint16_t* Bs = b_buf(st);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if constexpr (L::kAK) fa[set][i] = frag_k(As, TM, wm * (TM / 2) + 32 * i, kk);
      else fa[set][i] = frag_r(As, wm * (TM / 2) + 32 * i, kk);
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if constexpr (L::kBK) fb[set][j] = frag_k(Bs, kTgN, 64 * wn + 32 * j, kk);
      else fb[set][j] = frag_r(Bs, 64 * wn + 32 * j, kk);
    }
  };
  auto mma = [&](int set) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[set][i], fb[set][j], acc[i][j], 0, 0, 0);
  };
  // the next k-step's reads one by one between this k-step's MFMAs
  auto order = [&]() {
    constexpr int nr = MI * (L::kAK ? 2 : 1) + NJ * (L::kBK ? 2 : 1), nm = MI * NJ;
    if constexpr (nm >= nr) {
      constexpr int per = nm / nr, left = nm - nr * per;
#pragma unroll
      for (int q = 0; q < nr; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, per, 0);
      }
      if constexpr (left > 0) __builtin_amdgcn_sched_group_barrier(0x008, left, 0);
    } else {
      constexpr int per = nr / nm, left = nr - nm * per;
#pragma unroll
      for (int q = 0; q < nm; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x100, per, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      }
      if constexpr (left > 0) __builtin_amdgcn_sched_group_barrier(0x100, left, 0);
    }
  };
  auto mma_copies = [&](int set, int cst, int first, int cnt, bool on, auto of_slab) {
    constexpr int nm = MI * NJ;
#pragma unroll
    for (int q = 0; q < nm; ++q) {
      acc[q / NJ][q % NJ] =
          __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[set][q / NJ], fb[set][q % NJ], acc[q / NJ][q % NJ], 0, 0, 0);
#pragma unroll
      for (int c = 0; c < cnt; ++c)
        if (on && (c * nm) / cnt == q) issue_one(cst, first + c, of_slab);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // On entry the fragments of k-step 0 are in set 0 and the copies of stage st + 1 are complete or in flight, as
  // are those of B of stage st + 2; its A tile goes out after this stage's barrier.
  auto stage = [&](int st, bool refill, bool next, auto of_slab) {
#pragma unroll
    for (int kk = 0; kk < kTgK / 16 - 1; ++kk) {
      frag(st, kk + 1, (kk + 1) & 1);
      if (kk == 1) {
        mma_copies(1, st + 2, NA, NB, refill, of_slab);
      } else {
        mma(kk & 1);
        order();
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (refill) asm volatile("s_waitcnt vmcnt(%0)" :: "n"(NB) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    if (next) frag(st + 1, 0, 0);
    mma_copies(1, st + 2, 0, NA, refill, of_slab);
  };
  auto issue = [&](int st) {
    if (L::kSlab && s0 + st >= nmain) {
#pragma unroll
      for (int q = 0; q < NA + NB; ++q) issue_one(st, q, std::true_type{});
    } else {
#pragma unroll
      for (int q = 0; q < NA + NB; ++q) issue_one(st, q, std::false_type{});
    }
  };
  if (nk > 0) issue(0);
  if (nk > 1) issue(1);
  if (nk > 0) {
    if (nk > 1) asm volatile("s_waitcnt vmcnt(%0)" :: "n"(NA + NB) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    frag(0, 0, 0);
  }
  int st = 0;
  const int nm = nmain - s0 < nk ? nmain - s0 : nk;  // main stages of the slice (none: <= 0)
  for (; st + 2 < nm; ++st) stage(st, true, true, std::false_type{});
  if constexpr (L::kSlab) {
    for (; st + 2 < nk; ++st) stage(st, true, true, std::true_type{});
  }
  if (st + 1 < nk) stage(st++, false, true, std::false_type{});
  if (st < nk) stage(st, false, false, std::false_type{});
  __syncthreads();
  epi.template operator()<MI>(acc, m0, n0, wm, wn, z, smem);
}

// How a launch's tiles cover M x N on `cus` compute units, one workgroup each at a time: tiles of 256 or 128 rows and
// slices of the reduction of nk stages, whichever end soonest. A stage of a half-height tile took 1.0 us beside 1.65 of
// a full one (products of 6144 rows). Slices' partials are written and read once (S M N 8 bytes at 4.5 TB/s) and take
// one launch more; at least 8 stages each, at most 16, and M S at most `most` rows of partials. P W of 777 rows, 4096
// columns, 501 stages, both in short runs: half tiles in 2 slices 264 us, full ones in 4 214 (now, in long runs, 162). In fp32 arithmetic, on the host or the device
// (where M may be known there only: then of the choices that `grid` workgroups hold; whole tiles without slices have to
// be one).
constexpr float kTgFullCost = 1.65f, kTgHalfCost = 1.05f;

struct TgPlan {
  int tiles_m, tiles_n, half;     // half: tiles of 128 rows
  int slices, per_slice;
};

// Time of S slices in full or half-height tiles (*half), whichever is less; 3e38 where there may be no S slices.
__host__ __device__ inline float tg_cost(int64_t M, int64_t N, int nk, int64_t most, int cus, int grid, int S, bool* half) {
  const int t1 = (int)((M + 255) / 256), t2 = (int)((M + 127) / 128), tn = (int)((N + kTgN - 1) / kTgN);
  const int per = (nk + S - 1) / S;
  if (S > 1 && (nk < 8 * S || S * M > most || (nk + per - 1) / per != S)) return 3e38f;   // the last: a slice would be empty
  const float f1 = (float)t1 * tn / cus, f2 = (float)t2 * tn / cus, join = 8e-6f / 4.5f * M * N;
  const float f = (float)t1 * tn * S <= grid ? kTgFullCost * __builtin_ceilf(f1 * S) : 3e38f;
  const float h = (float)t2 * tn * S <= grid ? kTgHalfCost * __builtin_ceilf(f2 * S) : 3e38f;
  *half = h < f;
  return per * (f < h ? f : h) + (S > 1 ? 3.0f + join * S : 0.0f);
}

__host__ __device__ inline TgPlan tg_plan_of(int64_t M, int64_t N, int nk, int S, bool half) {
  const int rows = half ? 128 : 256;
  return TgPlan{(int)((M + rows - 1) / rows), (int)((N + kTgN - 1) / kTgN), half ? 1 : 0, S, (nk + S - 1) / S};
}

inline TgPlan tg_plan(int64_t M, int64_t N, int nk, int64_t most, int cus, int grid = 0x7FFFFFFF) {
  int best = 1;
  bool half = false;
  float least = 3e38f;
  for (int S = 1; S <= 16; ++S) {
    bool h = false;
    const float t = tg_cost(M, N, nk, most, cus, grid, S, &h);
    if (t < least) {
      least = t;
      best = S;
      half = h;
    }
  }
  return tg_plan_of(M, N, nk, best, half);
}

// The same by a wave, a slice count per lane (one after the other they took 2 us); every lane gets it.
__device__ inline TgPlan tg_plan_wave(int64_t M, int64_t N, int nk, int64_t most, int cus, int grid) {
  const int lane = threadIdx.x & 63;
  bool h = false;
  float t = lane < 16 ? tg_cost(M, N, nk, most, cus, grid, lane + 1, &h) : 3e38f;
  int best = 2 * lane + (h ? 1 : 0);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {                  // of equal times the fewest slices
    const float ot = __shfl_xor(t, o, 64);
    const int ob = __shfl_xor(best, o, 64);
    if (ot < t || (ot == t && ob < best)) {
      t = ot;
      best = ob;
    }
  }
  best = __builtin_amdgcn_readfirstlane(best);
  return tg_plan_of(M, N, nk, (best >> 1) + 1, best & 1);
}

// The same without slices, in a few integer operations: every workgroup of a product makes it for itself.
__host__ __device__ inline TgPlan tg_plan1(int64_t M, int64_t N, int nk, int cus, int grid = 0x7FFFFFFF) {
  const uint32_t t1 = (uint32_t)((M + 255) / 256), t2 = (uint32_t)((M + 127) / 128), tn = (uint32_t)((N + kTgN - 1) / kTgN);
  const uint32_t full = (t1 * tn + cus - 1) / cus, half = (t2 * tn + cus - 1) / cus;
  const bool h = 165 * full > 105 * half && t2 * tn <= (uint32_t)grid;
  return TgPlan{(int)(h ? t2 : t1), (int)tn, h ? 1 : 0, 1, nk};
}

// Rows of partials (slices times M) that a product of M rows may take: 16 slices of few rows, two of many, none of so
// many that two whole slices would not run sooner. Never fewer for more rows: a workspace for M rows serves fewer.
inline int64_t tg_partial_rows(int64_t M) {
  const int64_t m = M < 32768 ? M : 32768, few = 16 * m < 8192 ? 16 * m : 8192;
  return few > 2 * m ? few : 2 * m;
}

// A grid for plans of any M' <= M that are made on the device: that of M itself, and three rounds where slices or
// half-height tiles can use them.
inline int tg_grid(int64_t M, int64_t N, int nk, int64_t most, int cus) {
  const TgPlan p = tg_plan(M, N, nk, most, cus);
  const int64_t n = (int64_t)p.tiles_m * p.tiles_n * p.slices;
  const int64_t all = ((M + 127) / 128) * p.tiles_n * (most > 0 ? 16 : 1), more = all < 3 * cus ? all : 3 * cus;
  return (int)(n > more ? n : more);
}

// fp32 partials of a tile, straight from the accumulators (128-byte rows per half wave).
template <int MI>
__device__ __forceinline__ void tg_store_partial(f32x16_t (&acc)[MI][2], float* out, int64_t M, int64_t N, int64_t m0,
                                                 int64_t n0, int wm, int wn) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int64_t row = m0 + wm * (32 * MI) + 32 * i + (v & 3) + 4 * (lane >> 5) + 8 * (v >> 2);
      if (row >= M) continue;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t col = n0 + 64 * wn + 32 * j + (lane & 31);
        if (col < N) out[row * N + col] = acc[i][j][v];
      }
    }
}

// Tile and slice of workgroup bid: each of the 8 XCDs (bid % 8) takes a contiguous
// range of the tiles, ordered in groups of 4 tile-rows, so that concurrent tiles
// share rows of A and columns of B in one L2.
__device__ __forceinline__ bool tg_where(const TgPlan& pl, int bid, int64_t* m0, int64_t* n0, int* z) {
  const int per = pl.tiles_m * pl.tiles_n, n = per * pl.slices;
  if (bid >= n) return false;
  const int xcd = bid % 8, q = n / 8, rem = n % 8;
  const int w = xcd * q + (xcd < rem ? xcd : rem) + bid / 8;
  *z = w / per;
  const int t = w - *z * per;
  const int g = t / (4 * pl.tiles_n), first = 4 * g;
  const int gm = pl.tiles_m - first < 4 ? pl.tiles_m - first : 4;
  const int tl = t - g * 4 * pl.tiles_n;
  *m0 = (int64_t)(first + tl % gm) * (pl.half ? 128 : 256);
  *n0 = (int64_t)(tl / gm) * kTgN;
  return true;
}

// The workgroup's tile of a plan.
template <class L, class E>
__device__ __forceinline__ void tg_run(TgArgs& p, const E& epi, const TgPlan& pl, uint16_t* smem) {
  p.per_slice = pl.per_slice;
  int64_t m0, n0;
  int z;
  if (!tg_where(pl, (int)blockIdx.x, &m0, &n0, &z)) return;
  if (pl.half) tg_tile<128, L>(p, epi, m0, n0, smem, z);
  else tg_tile<256, L>(p, epi, m0, n0, smem, z);
}

}  // namespace qlora
