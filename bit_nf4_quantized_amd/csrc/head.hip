// Softmax cross entropy over a large vocabulary from hidden states H [M][K] and
// the head's weight W [V][K], without the logits S = H W^T in memory, and its
// gradients, for gfx950:
//
//   nll_m = log sum_v exp(S_mv) - S_my,   y = labels[m];   loss = sum_m w_m nll_m / divisor
//   dH_m = g_m (sum_v p_mv W_v - W_y),   dW_v = sum_m g_m (p_mv - [v = y]) H_m,   g_m = grad_scale w_m / divisor
//
// The exponentials are taken against the row's own label logit, which a dot
// product per row gives beforehand: with P_mv = exp(S_mv - S_my) for v != y and
// l_m = sum of them, nll = log(1 + l), p_mv = P_mv / (1 + l), and the label's
// gradient p_my - 1 = -l / (1 + l) has no cancellation. So no pass for the row's
// maximum is needed: P goes to bf16 (whose exponents are fp32's) straight from the
// logits' accumulators, with one rounding, and dH is one product of P with W, its
// rows scaled by g / (1 + l) at the end. A label with less than about e^-40 of the
// largest probability would let P overflow: where a logit of a 256-column tile is
// more than 40 above the label's, the tile takes its row's maximum out (its shift),
// and the rows' statistics bring the tiles to one shift.
//
//   head_rows_kernel     the list of counted rows (one workgroup; labels outside [0, V) do not count)
//   head_gather_kernel   their rows of H side by side, their label logits; zero rows of dH for the others
//   head_prob_kernel     the GEMM H W^T in 256 x 256 tiles, P and the tiles' row sums from its accumulators
//   head_stat_kernel     l, nll, the rows' scales; P_my = -l
//   head_dw_kernel       the GEMM P^T (scale H), both operands read down their rows
//   head_dh_kernel       the GEMM P W, W read down its rows, in slices of the vocabulary where that fills the device better
//   head_dh_sum_kernel   the slices' sum; the loss, a weighted sum in fp64
// In long runs of calls, 6144 counted rows x 4096 x 32000: P 1292-1364 us and dH 1187-1281 (1.18-1.36 PFLOP/s; a large
// library product 1.46), dW 1318-1372, the rest 85. 48 rows: P 64 us, 64 stages of 1.0 us on 125 of the 256 CUs; dH 46,
// bound by reading W (5.6 TB/s). 700 rows of 32001 with dW: P 194 us (750 half-height tiles, 2.9 rounds), dH 162, dW
// 194-202 (11 stages a tile, its stores 26 of them).
// Rows are taken in pieces whose P fits a gigabyte, but of 256 rows at least (2 GB of P at 2^22 words). The number of
// counted rows is known on the device only: the GEMMs plan their tiles there, from a grid for all rows. Without a
// gradient P is neither stored nor given room: the product's epilogue keeps the tiles' sums.
#include "common.h"
#include "launch.h"
#include "tile_gemm.h"

namespace qlora {

namespace {

int64_t hd_cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr float kShiftAbove = 40.0f;

// ---- rows --------------------------------------------------------------------------------

// rows[0 .. count): the counted rows in order; slot[m]: a row's place among them, or -1.
__global__ __launch_bounds__(1024) void head_rows_kernel(const int64_t* __restrict__ labels, int64_t M, int64_t V,
                                                         int32_t* __restrict__ rows, int32_t* __restrict__ slot,
                                                         int32_t* __restrict__ count) {
  __shared__ int s_n[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int n = 0;
  for (int64_t base = 0; base < M; base += 1024) {
    const int64_t m = base + tid;
    const int64_t y = m < M ? labels[m] : -1;
    const bool on = y >= 0 && y < V;
    const unsigned long long b = __ballot(on);
    if (lane == 0) s_n[wave] = __popcll(b);
    __syncthreads();
    int before = n, all = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      before += w < wave ? s_n[w] : 0;
      all += s_n[w];
    }
    const int at = before + __popcll(b & ((1ull << lane) - 1ull));
    if (on) rows[at] = (int32_t)m;
    if (m < M) slot[m] = on ? at : -1;
    n += all;
    __syncthreads();
  }
  if (tid == 0) count[0] = n;
}

struct HeadRows {
  const int32_t* rows;
  const int32_t* count;
  const float* ref;       // the exponentials' reference: the label's logit (0 where that is not finite)
  const float* logit;     // the label's logit
  const int32_t* label;
};

// FEW (up to kFewRows rows): each workgroup counts the rows before its own itself, and the last one writes the count:
// one launch less (48 rows: 10.2 -> 5.2 us).
constexpr int64_t kFewRows = 2048;

template <bool FEW>
__global__ __launch_bounds__(256) void head_gather_kernel(const uint16_t* __restrict__ H, const uint16_t* __restrict__ W,
                                                          const int64_t* __restrict__ labels, int64_t K, int64_t M, int64_t V,
                                                          int32_t* __restrict__ rows, int32_t* __restrict__ count,
                                                          const int32_t* __restrict__ slot, uint16_t* __restrict__ Hc,
                                                          float* __restrict__ ref, float* __restrict__ logit,
                                                          int32_t* __restrict__ label, float* __restrict__ nll,
                                                          uint16_t* __restrict__ dH) {
  __shared__ float red[4];
  const int64_t m = blockIdx.x;
  int at;
  if constexpr (FEW) {
    __shared__ int s_n[4];
    int n = 0;                                      // counted rows up to this one
    for (int64_t i = threadIdx.x; i <= m; i += 256) {
      const int64_t y = labels[i];
      n += y >= 0 && y < V;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o, 64);
    if ((threadIdx.x & 63) == 0) s_n[threadIdx.x >> 6] = n;
    __syncthreads();
    n = (s_n[0] + s_n[1]) + (s_n[2] + s_n[3]);
    const int64_t y = labels[m];
    at = y >= 0 && y < V ? n - 1 : -1;
    if (threadIdx.x == 0) {
      if (at >= 0) rows[at] = (int32_t)m;
      if (m == M - 1) count[0] = n;
    }
  } else {
    at = slot[m];
  }
  if (at < 0) {
    if (threadIdx.x == 0) nll[m] = 0.0f;
    if (dH)
      for (int64_t k = threadIdx.x * 8; k < K; k += 2048) *reinterpret_cast<u32x4_t*>(dH + m * K + k) = u32x4_t{0u, 0u, 0u, 0u};
    return;
  }
  const int64_t y = labels[m];
  float sum = 0.0f;
  for (int64_t k = threadIdx.x * 8; k < K; k += 2048) {
    const u32x4_t h = *reinterpret_cast<const u32x4_t*>(H + m * K + k), w = *reinterpret_cast<const u32x4_t*>(W + y * K + k);
    *reinterpret_cast<u32x4_t*>(Hc + (int64_t)at * K + k) = h;
    const uint32_t a[4] = {h.x, h.y, h.z, h.w}, b[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sum = __builtin_fmaf(__uint_as_float(a[e] << 16), __uint_as_float(b[e] << 16), sum);
      sum = __builtin_fmaf(__uint_as_float(a[e] & 0xFFFF0000u), __uint_as_float(b[e] & 0xFFFF0000u), sum);
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = (red[0] + red[1]) + (red[2] + red[3]);
    logit[at] = sum;
    ref[at] = __builtin_isfinite(sum) ? sum : 0.0f;
    label[at] = (int32_t)y;
  }
}

// Rows of a piece that starts at row0: how many there are.
__device__ __forceinline__ int64_t piece_rows(const int32_t* count, int64_t row0, int64_t piece) {
  const int64_t n = (int64_t)__builtin_amdgcn_readfirstlane(count[0]) - row0;
  return n < 0 ? 0 : n < piece ? n : piece;
}

// ---- P -----------------------------------------------------------------------------------

__device__ __forceinline__ float sum16(float v) {   // over each 16 lanes, in every lane
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, false));   // quad_perm 1,0,3,2
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, false));   // quad_perm 2,3,0,1
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xF, 0xF, false));  // row_half_mirror
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x140, 0xF, 0xF, false));  // row_mirror
  return v;
}

__device__ __forceinline__ float max16(float v) {
  v = __builtin_fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, false)));
  v = __builtin_fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, false)));
  v = __builtin_fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xF, 0xF, false)));
  v = __builtin_fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x140, 0xF, 0xF, false)));
  return v;
}

// P (STORE) and the tile's sums and shifts [tile][piece]. Columns from V on and rows past the counted ones: zeros.
template <bool STORE>
struct ProbEpi {
  const float* ref;       // of the piece's first row
  const int32_t* label;
  int64_t rows;           // counted rows of the piece
  int64_t V, ldp, piece;
  uint16_t* P;
  float* sum;
  float* shift;
  template <int MI>
  __device__ __forceinline__ void operator()(f32x16_t (&acc)[MI][2], int64_t m0, int64_t n0, int wm, int wn, int z,
                                             uint16_t* smem) const {
    constexpr int TM = 64 * MI;
    const int tid = threadIdx.x, lane = tid & 63;
    float* s_ref = reinterpret_cast<float*>(smem);
    int* s_label = reinterpret_cast<int*>(s_ref + 256);
    float* s_shift = s_ref + 512;
    float* s_part = s_ref + 768;                    // [8][256]
    int* s_over = reinterpret_cast<int*>(s_ref + 768 + 2048);
    uint16_t* ep = smem + 2 * (768 + 2048 + 64) + (wm * 4 + wn) * (32 * 72);
    if (tid == 0) *s_over = 0;
    if (tid < TM) {
      const bool in = m0 + tid < rows;
      s_ref[tid] = in ? ref[m0 + tid] : 0.0f;
      s_label[tid] = in ? (int)(label[m0 + tid] - n0) : -1;    // column in the tile
      s_shift[tid] = 0.0f;
    }
    __syncthreads();
    const int c0 = 64 * wn + (lane & 31);
    const bool in0 = n0 + c0 < V, in1 = n0 + c0 + 32 < V;
    auto row_of = [&](int i, int v) { return wm * (32 * MI) + 32 * i + (v & 3) + 4 * (lane >> 5) + 8 * (v >> 2); };
    bool over = false;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int r = row_of(i, v);
        const float f = s_ref[r];
        const int y = s_label[r];
        const bool live = m0 + r < rows;
        // masked entries: -inf, whose exponential is 0
        acc[i][0][v] = live && in0 && c0 != y ? acc[i][0][v] - f : -__builtin_inff();
        acc[i][1][v] = live && in1 && c0 + 32 != y ? acc[i][1][v] - f : -__builtin_inff();
        over = over || acc[i][0][v] > kShiftAbove || acc[i][1][v] > kShiftAbove;
      }
    if (__any(over) && lane == 0) *s_over = 1;
    __syncthreads();
    if (*s_over) {                                  // uniform
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const float m = max16(__builtin_fmaxf(acc[i][0][v], acc[i][1][v]));
          if ((lane & 15) == 0) s_part[(2 * wn + ((lane >> 4) & 1)) * 256 + row_of(i, v)] = m;
        }
      __syncthreads();
      if (tid < TM) {
        float m = s_part[tid];
#pragma unroll
        for (int q = 1; q < 8; ++q) m = __builtin_fmaxf(m, s_part[q * 256 + tid]);
        s_shift[tid] = m > kShiftAbove ? m : 0.0f;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const float d = s_shift[row_of(i, v)];
          acc[i][0][v] -= d;
          acc[i][1][v] -= d;
        }
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      float mine = 0.0f;                            // of the lane's row: register v = lane % 16
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const float a = __expf(acc[i][0][v]), b = __expf(acc[i][1][v]);
        const float s = sum16(a + b);
        mine = (lane & 15) == v ? s : mine;
        if constexpr (STORE) {
          const int at = ((v & 3) + 4 * (lane >> 5) + 8 * (v >> 2)) * 72 + (lane & 31);
          ep[at] = f32_to_bf16(a);
          ep[at + 32] = f32_to_bf16(b);
        }
      }
      {
        const int v = lane & 15;
        s_part[(2 * wn + ((lane >> 4) & 1)) * 256 + row_of(i, v)] = mine;
      }
      if constexpr (STORE) {
        __builtin_amdgcn_s_waitcnt(0xc07f);         // lgkmcnt(0): the wave's own slice
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const int r = 8 * it + (lane >> 3), c = 8 * (lane & 7);
          const u32x4_t val = *reinterpret_cast<const u32x4_t*>(ep + r * 72 + c);
          const int64_t row = m0 + wm * (32 * MI) + 32 * i + r, col = n0 + 64 * wn + c;
          if (row < piece && col < ldp) *reinterpret_cast<u32x4_t*>(P + row * ldp + col) = val;
        }
        __builtin_amdgcn_s_waitcnt(0xc07f);
      }
    }
    __syncthreads();
    if (tid < TM && m0 + tid < rows) {
      float s = s_part[tid];
#pragma unroll
      for (int q = 1; q < 8; ++q) s += s_part[q * 256 + tid];
      const int64_t at = (n0 / kTgN) * piece + m0 + tid;
      sum[at] = s;
      shift[at] = s_shift[tid];
    }
  }
};

template <bool STORE>
__global__ __launch_bounds__(kTgThreads, 1) void head_prob_kernel(TgArgs p, ProbEpi<STORE> epi, const int32_t* count, int64_t row0,
                                                                  int64_t N, int cus) {
  __shared__ __attribute__((aligned(1024))) uint16_t smem[kTgSmem];
  epi.rows = piece_rows(count, row0, epi.piece);
  tg_run<TgLayout<false, false, false, false>>(p, epi, tg_plan1(epi.rows, N, (int)(p.kmain / kTgK), cus, (int)gridDim.x), smem);
}

// ---- statistics ----------------------------------------------------------------------------

// 64 rows per workgroup, one per lane; wave w joins the tiles w, w + 16, ... with its rows' sums, then the waves in
// order. A row's tiles are brought to its largest shift D: l = sum_t sum_t e^(shift_t - D), and with e_y = e^-D
// (0 where the label's logit is -inf) nll = D + log(e_y + l) (+ reference - label's logit) and scale = g / (e_y + l).
struct StatArgs {
  const float* sum;
  const float* shift;
  int tiles;
  int64_t row0, piece, ldp;
  HeadRows r;
  const float* weights;
  float divisor, grad_scale;
  uint16_t* P;             // nullptr: the loss alone
  float* scale;            // of the piece
  float* nll;              // by row
  TgPlan* plan;            // of P W, made by the first workgroup; nullptr: no dH
  int64_t K, most;         // its columns, its rows of partials at most
  int nk, cus, grid;
};

__global__ __launch_bounds__(1024) void head_stat_kernel(StatArgs a) {
  __shared__ float s_d[16][64], s_l[16][64], s_top[64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t n = piece_rows(a.r.count, a.row0, a.piece), r0 = (int64_t)blockIdx.x * 64;
  if (a.plan && r0 == 0 && wave == 15) {
    const TgPlan pl = tg_plan_wave(n, a.K, a.nk, a.most, a.cus, a.grid);
    if (lane == 0) *a.plan = pl;
  }
  if (r0 >= n) return;                              // uniform
  const bool in = r0 + lane < n;
  const int64_t row = in ? r0 + lane : n - 1;
  float d = 0.0f, l = 0.0f;
  bool moved = false;
  constexpr int kBatch = 8;                         // tiles whose loads are in flight
  for (int t0 = wave; t0 < a.tiles; t0 += 16 * kBatch) {
    float sv[kBatch], hv[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int64_t t = t0 + 16 * u < a.tiles ? t0 + 16 * u : t0;
      sv[u] = a.sum[t * a.piece + row];
      hv[u] = a.shift[t * a.piece + row];
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (t0 + 16 * u >= a.tiles) break;            // uniform
      const float s = sv[u], h = hv[u];
      moved = moved || h != 0.0f;
      if (h > d) {
        l *= __expf(d - h);
        d = h;
      }
      l += h == d ? s : s * __expf(h - d);
    }
  }
  s_d[wave][lane] = d;
  s_l[wave][lane] = l;
  __syncthreads();
  d = s_d[0][lane];
#pragma unroll
  for (int w = 1; w < 16; ++w) d = __builtin_fmaxf(d, s_d[w][lane]);
  l = 0.0f;
#pragma unroll
  for (int w = 0; w < 16; ++w) l += s_d[w][lane] == d ? s_l[w][lane] : s_l[w][lane] * __expf(s_d[w][lane] - d);
  const int64_t at = a.row0 + row;
  if (wave == 0) {
    const float logit = a.r.logit[at], ref = a.r.ref[at];
    const float ey = logit == ref ? __expf(-d) : __expf(logit);   // reference 0: e^-inf = 0, or not a number
    const float total = ey + l;
    const int32_t m = a.r.rows[at];
    const float nll = (logit == ref && d == 0.0f ? log1pf(l) : d + __logf(total)) + (ref - logit);
    const float w = a.weights ? a.weights[m] : 1.0f;
    const float div = a.divisor != 0.0f ? a.divisor : (float)a.r.count[0];
    const float scale = a.grad_scale * w / div / total;
    s_top[lane] = d;
    if (in) {
      a.nll[m] = nll;
      a.scale[row] = scale;
    }
  }
  if (!a.P) return;
  __syncthreads();
  const bool any = __syncthreads_or(moved || d != 0.0f);
  if (any) {                                        // rare: rows whose tiles have different shifts
    for (int q = 0; q < 64 && r0 + q < n; ++q) {
      const float top = s_top[q];
      if (top == 0.0f) continue;
      uint16_t* p = a.P + (r0 + q) * a.ldp;
      for (int64_t c = tid; c < a.ldp; c += 1024) {
        const float h = a.shift[(c / kTgN) * a.piece + r0 + q];
        if (h != top) p[c] = f32_to_bf16(bf16_to_f32(p[c]) * __expf(h - top));
      }
    }
    __syncthreads();
  }
  if (wave == 0 && in) a.P[row * a.ldp + a.r.label[at]] = f32_to_bf16(-l);
}

// dW's operand: the piece's rows of H, scaled.
__global__ __launch_bounds__(256) void head_scale_kernel(uint16_t* __restrict__ Hc, const float* __restrict__ scale,
                                                         const int32_t* count, int64_t row0, int64_t piece, int64_t K) {
  const int64_t n = piece_rows(count, row0, piece), per = K / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n * per; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per;
    uint16_t* h = Hc + i * 8;
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(h);
    const float s = scale[row];
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = pack_bf16x2(s * __uint_as_float(x[e] << 16), s * __uint_as_float(x[e] & 0xFFFF0000u));
    *reinterpret_cast<u32x4_t*>(h) = u32x4_t{o[0], o[1], o[2], o[3]};
  }
}

// ---- gradients --------------------------------------------------------------------------------

// dH rows, scaled, at their places; or, in reduction slices, fp32 partials [slices][n][K].
struct DhEpi {
  const float* scale;      // of the piece
  const int32_t* rows;
  int64_t n, K, piece;
  uint16_t* dH;
  float* part;             // nullptr: one slice
  template <int MI>
  __device__ __forceinline__ void operator()(f32x16_t (&acc)[MI][2], int64_t m0, int64_t n0, int wm, int wn, int z,
                                             uint16_t* smem) const {
    const int lane = threadIdx.x & 63;
    if (part) {
      tg_store_partial(acc, part + (int64_t)z * n * K, n, K, m0, n0, wm, wn);
      return;
    }
    constexpr int kPitch = 64 + 8;
    uint16_t* ep = smem + (wm * 4 + wn) * (32 * kPitch);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int r = (v & 3) + 4 * (lane >> 5) + 8 * (v >> 2);
        const int64_t row = m0 + wm * (32 * MI) + 32 * i + r;
        const float s = scale[row < n ? row : n - 1];
#pragma unroll
        for (int j = 0; j < 2; ++j) ep[r * kPitch + 32 * j + (lane & 31)] = f32_to_bf16(s * acc[i][j][v]);
      }
      __builtin_amdgcn_s_waitcnt(0xc07f);
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int r = 8 * it + (lane >> 3), c = 8 * (lane & 7);
        const u32x4_t val = *reinterpret_cast<const u32x4_t*>(ep + r * kPitch + c);
        const int64_t row = m0 + wm * (32 * MI) + 32 * i + r, col = n0 + 64 * wn + c;
        if (row < n && col < K) *reinterpret_cast<u32x4_t*>(dH + (int64_t)rows[row] * K + col) = val;
      }
      __builtin_amdgcn_s_waitcnt(0xc07f);
    }
  }
};

__global__ __launch_bounds__(kTgThreads, 1) void head_dh_kernel(TgArgs p, DhEpi epi, const int32_t* count, int64_t row0,
                                                                const TgPlan* __restrict__ plan) {
  __shared__ __attribute__((aligned(1024))) uint16_t smem[kTgSmem];
  epi.n = piece_rows(count, row0, epi.piece);
  const TgPlan pl = *plan;
  if (pl.slices == 1) epi.part = nullptr;
  tg_run<TgLayout<false, true, false, false>>(p, epi, pl, smem);
}

// The weighted sum of the rows' losses, in fp64 and in a fixed order; the whole workgroup.
struct LossArgs {
  const float* nll;
  const float* weights;
  const int32_t* rows;
  const int32_t* count;
  float divisor;
  float* loss;
};

__device__ __forceinline__ void head_loss_body(const LossArgs& a) {
  __shared__ double red[4];
  const int n = a.count[0], tid = threadIdx.x;
  double s = 0.0;
  for (int i = tid; i < n; i += 1024) {              // 4 rows' loads in flight
    int32_t m[4];
    float v[4], w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) m[u] = a.rows[i + 256 * u < n ? i + 256 * u : i];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      v[u] = a.nll[m[u]];
      w[u] = a.weights ? a.weights[m[u]] : 1.0f;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + 256 * u < n) s += (double)v[u] * (double)w[u];
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
  if ((tid & 63) == 0) red[tid >> 6] = s;
  __syncthreads();
  if (tid == 0) {
    s = (red[0] + red[1]) + (red[2] + red[3]);
    const double div = a.divisor != 0.0f ? (double)a.divisor : (double)(n > 0 ? n : 1);
    a.loss[0] = (float)(s / div);
  }
}

__global__ __launch_bounds__(256) void head_loss_kernel(LossArgs a) { head_loss_body(a); }

// dH from its slices, added in order, 8 loads in flight; in the last piece, the last workgroup sums the loss.
__global__ __launch_bounds__(256) void head_dh_sum_kernel(const float* __restrict__ part, const TgPlan* __restrict__ plan, int64_t piece,
                                                          int64_t K, int64_t row0, const float* __restrict__ scale,
                                                          const int32_t* __restrict__ rows, uint16_t* __restrict__ dH, LossArgs la) {
  if (blockIdx.x == gridDim.x - 1) {
    if (la.loss) head_loss_body(la);
    return;
  }
  const int S = plan->slices;
  if (S == 1) return;
  const int64_t n = piece_rows(la.count, row0, piece), per = K / 8, step = n * K;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n * per; i += (int64_t)(gridDim.x - 1) * 256) {
    const int64_t row = i / per, k = (i - row * per) * 8;
    const float* q = part + i * 8;
    f32x4_t a = {0.0f, 0.0f, 0.0f, 0.0f}, b = a;
    for (int z = 0; z < S; z += 4) {
      f32x4_t u[4], v[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float* o = q + (z + t < S ? z + t : z) * step;
        u[t] = *reinterpret_cast<const f32x4_t*>(o);
        v[t] = *reinterpret_cast<const f32x4_t*>(o + 4);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (z + t >= S) break;                       // uniform
        a += u[t];
        b += v[t];
      }
    }
    const float s = scale[row];
    *reinterpret_cast<u32x4_t*>(dH + (int64_t)rows[row] * K + k) = u32x4_t{
        pack_bf16x2(s * a.x, s * a.y), pack_bf16x2(s * a.z, s * a.w), pack_bf16x2(s * b.x, s * b.y), pack_bf16x2(s * b.z, s * b.w)};
  }
}

// dW tile, with the sum of the pieces before in E (fp32; nullptr: none), to fp32 or bf16.
struct DwEpi {
  const float* E;
  void* out;
  bool bf16;
  int64_t V, K;
  template <int MI>
  __device__ __forceinline__ void operator()(f32x16_t (&acc)[MI][2], int64_t m0, int64_t n0, int wm, int wn, int z,
                                             uint16_t* smem) const {
    constexpr int kPitch = 64 + 4;
    const int lane = threadIdx.x & 63;
    float* ep = reinterpret_cast<float*>(smem) + (wm * 4 + wn) * (32 * kPitch);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int r = (v & 3) + 4 * (lane >> 5) + 8 * (v >> 2);
#pragma unroll
        for (int j = 0; j < 2; ++j) ep[r * kPitch + 32 * j + (lane & 31)] = acc[i][j][v];
      }
      __builtin_amdgcn_s_waitcnt(0xc07f);
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int r = 8 * it + (lane >> 3), c = 8 * (lane & 7);
        f32x4_t a = *reinterpret_cast<const f32x4_t*>(ep + r * kPitch + c);
        f32x4_t b = *reinterpret_cast<const f32x4_t*>(ep + r * kPitch + c + 4);
        const int64_t row = m0 + wm * (32 * MI) + 32 * i + r, col = n0 + 64 * wn + c;
        if (row < V && col < K) {
          const int64_t at = row * K + col;
          if (E) {
            a += *reinterpret_cast<const f32x4_t*>(E + at);
            b += *reinterpret_cast<const f32x4_t*>(E + at + 4);
          }
          if (bf16) {
            *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(out) + at) =
                u32x4_t{pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y), pack_bf16x2(b.z, b.w)};
          } else {
            *reinterpret_cast<f32x4_t*>(static_cast<float*>(out) + at) = a;
            *reinterpret_cast<f32x4_t*>(static_cast<float*>(out) + at + 4) = b;
          }
        }
      }
      __builtin_amdgcn_s_waitcnt(0xc07f);
    }
  }
};

__global__ __launch_bounds__(kTgThreads, 1) void head_dw_kernel(TgArgs p, DwEpi epi, TgPlan pl, const int32_t* count, int64_t row0,
                                                                int64_t piece) {
  __shared__ __attribute__((aligned(1024))) uint16_t smem[kTgSmem];
  const int64_t n = piece_rows(count, row0, piece);
  p.kmain = (n + kTgK - 1) / kTgK * kTgK;           // P's rows up to there are zeros, H's repeat its last row
  p.krows_a = p.kmain > 0 ? p.kmain : 1;
  p.krows_b = n > 0 ? n : 1;
  pl.per_slice = (int)(p.kmain / kTgK);
  tg_run<TgLayout<true, true, false, false>>(p, epi, pl, smem);
}

__global__ __launch_bounds__(256) void head_zero_kernel(uint32_t* __restrict__ p, int64_t words) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words; i += (int64_t)gridDim.x * 256) p[i] = 0u;
}

// Rows of a piece: P of at most 2^29 values, at least 256 rows.
int64_t head_piece(int64_t M, int64_t ldp) {
  int64_t most = ((int64_t)1 << 29) / ldp / 256 * 256;
  if (most < 256) most = 256;
  const int64_t all = M > 256 ? hd_cdiv(M, 256) * 256 : 256;
  return all < most ? all : most;
}

}  // namespace

HeadWorkspace head_workspace_layout(int64_t M, int64_t K, int64_t V, bool dH, bool dW, bool dw_bf16) {
  const int64_t ldp = hd_cdiv(V, 64) * 64;
  HeadWorkspace L;
  L.piece = head_piece(M, ldp);
  size_t off = 0;
  auto take = [&](int64_t bytes) { const size_t at = off; off += align_up((size_t)bytes, 256); return at; };
  L.rows_off = take(8 * M);                         // rows, then slots
  L.count_off = take(4);
  L.ref_off = take(8 * M);                          // references, then label logits
  L.label_off = take(4 * M);
  L.scale_off = take(4 * L.piece);
  L.stat_off = take(8 * hd_cdiv(V, kTgN) * L.piece);
  L.h_off = take(2 * M * K);
  L.p_off = take(dH || dW ? 2 * L.piece * ldp : 0);
  L.most = dH ? tg_partial_rows(L.piece < M ? L.piece : M) : 0;
  L.part_off = take(4 * L.most * K);
  L.plan_off = take(sizeof(TgPlan));
  L.dw_off = take(dW && dw_bf16 && M > L.piece ? 4 * V * K : 0);
  L.total = off > 0 ? off : 256;
  return L;
}

hipError_t launch_head_loss(const HeadCall& c, hipStream_t stream) {
  const int64_t M = c.M, K = c.K, V = c.V, ldp = hd_cdiv(V, 64) * 64;
  const HeadWorkspace L = head_workspace_layout(M, K, V, c.dH != nullptr, c.dW != nullptr, c.dw_bf16);
  char* b = static_cast<char*>(c.ws);
  int32_t* rows = reinterpret_cast<int32_t*>(b + L.rows_off);
  int32_t* slot = rows + M;
  int32_t* count = reinterpret_cast<int32_t*>(b + L.count_off);
  float* ref = reinterpret_cast<float*>(b + L.ref_off);
  float* logit = ref + M;
  int32_t* label = reinterpret_cast<int32_t*>(b + L.label_off);
  float* scale = reinterpret_cast<float*>(b + L.scale_off);
  float* sum = reinterpret_cast<float*>(b + L.stat_off);
  const int64_t tiles = hd_cdiv(V, kTgN);
  float* shift = sum + tiles * L.piece;
  uint16_t* Hc = reinterpret_cast<uint16_t*>(b + L.h_off);
  uint16_t* P = reinterpret_cast<uint16_t*>(b + L.p_off);
  float* part = reinterpret_cast<float*>(b + L.part_off);
  float* dwsum = reinterpret_cast<float*>(b + L.dw_off);
  TgPlan* plan = reinterpret_cast<TgPlan*>(b + L.plan_off);
  const int cus = device_cu_count();
  const bool grad = c.dH || c.dW;

  if (M > 0 && M <= kFewRows) {
    hipLaunchKernelGGL(head_gather_kernel<true>, dim3((unsigned)M), dim3(256), 0, stream, c.H, c.W, c.labels, K, M, V, rows, count,
                       slot, Hc, ref, logit, label, c.nll, c.dH);
  } else {
    hipLaunchKernelGGL(head_rows_kernel, dim3(1), dim3(1024), 0, stream, c.labels, M, V, rows, slot, count);
    if (M > 0)
      hipLaunchKernelGGL(head_gather_kernel<false>, dim3((unsigned)M), dim3(256), 0, stream, c.H, c.W, c.labels, K, M, V, rows,
                         count, slot, Hc, ref, logit, label, c.nll, c.dH);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const HeadRows hr{rows, count, ref, logit, label};
  const LossArgs la{c.nll, c.weights, rows, count, c.divisor, c.loss};
  for (int64_t r0 = 0; r0 < M; r0 += L.piece) {
    const int64_t most = M - r0 < L.piece ? M - r0 : L.piece;     // rows there may be
    const bool last = r0 + L.piece >= M;
    TgArgs p{};
    p.A = {Hc + r0 * K, K, most};
    p.B = {c.W, K, V};
    p.kmain = K;
    const dim3 tiles_grid((unsigned)tg_grid(most, V, (int)(K / kTgK), 0, cus));
    if (grad)
      hipLaunchKernelGGL(head_prob_kernel<true>, tiles_grid, dim3(kTgThreads), 0, stream, p,
                         ProbEpi<true>{ref + r0, label + r0, 0, V, ldp, L.piece, P, sum, shift}, count, r0, V, cus);
    else
      hipLaunchKernelGGL(head_prob_kernel<false>, tiles_grid, dim3(kTgThreads), 0, stream, p,
                         ProbEpi<false>{ref + r0, label + r0, 0, V, ldp, L.piece, nullptr, sum, shift}, count, r0, V, cus);
    const int grid = tg_grid(most, K, (int)(ldp / kTgK), L.most, cus);
    const StatArgs sa{sum, shift, (int)tiles, r0, L.piece, ldp, hr, c.weights, c.divisor, c.grad_scale, grad ? P : nullptr,
                      scale, c.nll, c.dH ? plan : nullptr, K, L.most, (int)(ldp / kTgK), cus, grid};
    hipLaunchKernelGGL(head_stat_kernel, dim3((unsigned)hd_cdiv(most, 64)), dim3(1024), 0, stream, sa);
    if (c.dW) {
      const int64_t vectors = hd_cdiv(most * K / 8, 256);
      hipLaunchKernelGGL(head_scale_kernel, dim3((unsigned)(vectors < 16 * cus ? vectors : 16 * cus)), dim3(256), 0, stream,
                         Hc + r0 * K, scale, count, r0, L.piece, K);
      TgArgs q{};
      q.A = {P, ldp, ldp};
      q.B = {Hc + r0 * K, K, K};
      const TgPlan pl = tg_plan(V, K, (int)hd_cdiv(most, kTgK), 0, cus);
      float* f32 = c.dw_bf16 ? dwsum : static_cast<float*>(c.dW);
      const DwEpi we{r0 > 0 ? f32 : nullptr, last ? c.dW : f32, last && c.dw_bf16, V, K};
      hipLaunchKernelGGL(head_dw_kernel, dim3((unsigned)(pl.tiles_m * pl.tiles_n)), dim3(kTgThreads), 0, stream, q, we, pl, count, r0,
                         L.piece);
    }
    if (c.dH) {
      TgArgs q{};
      q.A = {P, ldp, L.piece};
      q.B = {c.W, K, K};
      q.kmain = ldp;
      q.krows_b = V;
      const DhEpi de{scale, rows + r0, 0, K, L.piece, c.dH, part};
      hipLaunchKernelGGL(head_dh_kernel, dim3((unsigned)grid), dim3(kTgThreads), 0, stream, q, de, count, r0, plan);
      LossArgs end = la;
      if (!last) end.loss = nullptr;
      int64_t blocks = hd_cdiv(most * K / 8, 256);
      if (blocks > 8 * cus) blocks = 8 * cus;
      hipLaunchKernelGGL(head_dh_sum_kernel, dim3((unsigned)blocks + 1), dim3(256), 0, stream, part, plan, L.piece, K, r0, scale,
                         rows + r0, c.dH, end);
    }
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (c.dW && M == 0) {
    const int64_t words = V * K / (c.dw_bf16 ? 2 : 1);
    hipLaunchKernelGGL(head_zero_kernel, dim3((unsigned)(4 * cus)), dim3(256), 0, stream, static_cast<uint32_t*>(c.dW), words);
  }
  if (!c.dH || M == 0) hipLaunchKernelGGL(head_loss_kernel, dim3(1), dim3(256), 0, stream, la);
  return hipGetLastError();
}

}  // namespace qlora
