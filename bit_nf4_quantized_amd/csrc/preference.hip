// Preference loss over pairs of sequences, with the gradient of the logits,
// for gfx950.
//
//   lp[s][t] = x[y] - lse(x),  x = logits[s][t][:], y = labels[s][t]
//   reward[s] = beta sum_{t counted} (lp[s][t] - ref[s][t]),  h_p = reward[p] - reward[P + p]
//   loss = mean_p (1 - eps) softplus(-h_p) + eps softplus(h_p)
//   dlogits[s][t][v] = w_s (onehot(y) - softmax(x))[v],
//   w_p = -g (beta / P) (sigmoid(-h_p) - eps),  w_{P+p} = -w_p,  g the gradient scale
// (a paired log-ratio loss: Rafailov et al., "Direct Preference Optimization",
// NeurIPS 2023, eq. 7, with label smoothing). A position whose label lies
// outside [0, V) does not count: its logits are not read and its gradient row
// is zero.
//
// Three kernels:
//   row_stats    one workgroup per counted row: one pass with a running
//                maximum and sum per thread, joined over the workgroup; writes
//                lp and the row's (maximum, 1 / sum)
//   pair_loss    one workgroup per pair: both rewards in float64 in a fixed
//                order, the pair's loss and gradient weight
//   row_grad     one workgroup per row: w (onehot - e^(x - max) / sum), one
//                rounding to the logits' type; may write over the logits. One
//                more workgroup adds the pairs' losses.
// The weight needs every row of its pair, so a counted logit is read twice and
// its gradient written once: both row kernels are bound by HBM. For 16
// sequences of 1024 x 32000 bf16 (72 % of the rows count: 0.75 GB read twice,
// 1.05 GB written) the call takes 0.45 ms, 5.6 TB/s, more than a large copy's rate:
// row_stats 133 us, pair_loss 5.5, row_grad 311.
// row_grad walks the rows backwards, so that the rows read last are still in
// the last-level cache, and stores past it (nontemporal): 0.50 ms without
// either, 0.495 ms with one of them, 0.47 with both. Launching both row kernels over groups of
// pairs that fit that cache was slower (0.54 ms for two groups, 0.62 ms for
// eight): each group adds three launches' ends.
// A row's first element need not be 16-byte aligned
// (odd vocabularies, odd strides): a workgroup handles the elements before
// the first aligned address and after the last one singly.
#include "common.h"
#include "launch.h"

namespace qlora {

namespace {

constexpr int kRowThreads = 256;
// log2(e) as a sum of two fp32: with the first alone every exponent would be
// off by 1.3e-8 of itself in one direction, and a sequence's sum of lp with it
constexpr float kLog2eHi = 1.44269502162933349609f;
constexpr float kLog2eLo = 1.92596299112661746887e-8f;

template <typename T> struct Vec;               // one 16-byte access
template <> struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const u32x4_t& w, float* x) {
    x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y); x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ u32x4_t pack(const float* x) {
    return u32x4_t{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
  }
  static __device__ __forceinline__ float one(float x) { return x; }
  static __device__ __forceinline__ float round(float x) { return x; }
};
template <> struct Vec<uint16_t> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const u32x4_t& w, float* x) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(v[i] << 16);
      x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ u32x4_t pack(const float* x) {
    return u32x4_t{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
  }
  static __device__ __forceinline__ float one(uint16_t x) { return bf16_to_f32(x); }
  static __device__ __forceinline__ uint16_t round(float x) { return f32_to_bf16(x); }
};

// A row as head singles, aligned 16-byte pieces, tail singles.
template <typename T>
struct RowParts {
  int head, pieces, tail0;    // tail singles from tail0 on
  __device__ __forceinline__ RowParts(const T* row, int V) {
    const int off = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    head = off ? Vec<T>::kN - off : 0;
    if (head > V) head = V;
    pieces = (V - head) / Vec<T>::kN;
    tail0 = head + pieces * Vec<T>::kN;
  }
};

// e^t for t <= 0 (0 for -inf)
__device__ __forceinline__ float exp_neg(float t) {
  return __builtin_amdgcn_exp2f(__builtin_fmaf(t, kLog2eHi, t * kLog2eLo));
}

// Running maximum and sum of e^(x - max). An empty sum has max = -inf, sum =
// 0; a maximum of -inf never enters an exponent (-inf minus -inf).
struct MaxSum {
  float m, s;
};

__device__ __forceinline__ MaxSum join(const MaxSum& a, const MaxSum& b) {
  const float m = __builtin_fmaxf(a.m, b.m);
  if (m == -__builtin_inff()) return MaxSum{m, a.s + b.s};
  return MaxSum{m, a.s * exp_neg(a.m - m) + b.s * exp_neg(b.m - m)};
}

template <int N>
__device__ __forceinline__ void fold(MaxSum& a, const float* x) {
  float top = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) top = __builtin_fmaxf(top, x[i]);
  if (top > a.m) {
    a.s *= exp_neg(a.m - top);    // a.m = -inf: 0
    a.m = top;
  }
  const float m = a.m == -__builtin_inff() ? 0.0f : a.m;
  float s = 0.0f;                 // the values' own sum first: a shorter chain of roundings
#pragma unroll
  for (int i = 0; i < N; ++i) s += exp_neg(x[i] - m);
  a.s += s;
}

struct PrefArgs {
  const void* x;            // logits [S T] rows of V, row stride ld elements
  const int64_t* labels;    // [S T]
  const float* ref;         // [S T]
  void* dx;                 // gradient, row stride ldd
  float* lp;                // [S T]
  f32x2_t* stat;            // [S T]: a row's maximum m and 1 / sum e^(x - m)
  double* pair;             // [S / 2]: a pair's loss
  float* w;                 // [S]
  float* reward;            // [S]
  float* loss;              // [1]
  int64_t rows;             // gradient rows
  int64_t ld, ldd;
  int S, T, V;
  float beta, eps, gscale;
};

// One workgroup per row, numbered over a grid of lines: one dimension of a
// launch holds fewer than 2^32 work-items, which 2^24 rows would reach.
// Workgroups past the last row end at once.
constexpr int64_t kRowsPerLine = 1 << 23;

dim3 row_grid(int64_t rows) {
  const int64_t line = rows < kRowsPerLine ? rows : kRowsPerLine;
  return dim3((unsigned)line, (unsigned)((rows + line - 1) / line));
}

__device__ __forceinline__ int64_t row_number() { return (int64_t)blockIdx.y * kRowsPerLine + blockIdx.x; }

template <typename T>
__global__ __launch_bounds__(kRowThreads) void row_stats_kernel(PrefArgs p) {
  __shared__ MaxSum part[kRowThreads / 64];
  const int tid = threadIdx.x;
  const int64_t row = row_number();
  if (row >= p.rows) return;                        // uniform: no barrier was reached
  const int64_t y = p.labels[row];
  if (y < 0 || y >= p.V) {
    if (tid == 0) p.lp[row] = 0.0f;
    return;
  }
  const T* x = static_cast<const T*>(p.x) + row * p.ld;
  const RowParts<T> r(x, p.V);
  constexpr int N = Vec<T>::kN;
  constexpr int kU = 8;
  MaxSum a = {-__builtin_inff(), 0.0f};
  if (tid < r.head) {
    const float v = Vec<T>::one(x[tid]);
    fold<1>(a, &v);
  }
  if (tid < p.V - r.tail0) {
    const float v = Vec<T>::one(x[r.tail0 + tid]);
    fold<1>(a, &v);
  }
  const u32x4_t* xv = reinterpret_cast<const u32x4_t*>(x + r.head);
  for (int b = tid; b < r.pieces; b += kU * kRowThreads) {
    u32x4_t raw[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int i = b + u * kRowThreads;
      raw[u] = xv[i < r.pieces ? i : b];
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float v[N];
      Vec<T>::unpack(raw[u], v);
      if (b + u * kRowThreads < r.pieces) fold<N>(a, v);
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    MaxSum b;
    b.m = __shfl_xor(a.m, o, 64);
    b.s = __shfl_xor(a.s, o, 64);
    a = join(a, b);
  }
  if ((tid & 63) == 0) part[tid >> 6] = a;
  __syncthreads();
  if (tid == 0) {
    a = part[0];
    for (int k = 1; k < kRowThreads / 64; ++k) a = join(a, part[k]);
    p.stat[row] = f32x2_t{a.m, 1.0f / a.s};
    p.lp[row] = (Vec<T>::one(x[y]) - a.m) - __builtin_logf(a.s);
  }
}

__device__ __forceinline__ double softplus(double z) { return (z > 0.0 ? z : 0.0) + log1p(exp(-fabs(z))); }

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// One workgroup per pair: half of the waves add the preferred sequence's
// positions in float64 (lane l of wave w: positions 64 w + l, + 512, ...), half
// the other's; then the lanes, then the waves. Latency-bound: 16 waves so that
// a sequence of some thousand positions is one or two round trips.
constexpr int kPairWaves = 16;

__global__ __launch_bounds__(64 * kPairWaves) void pair_loss_kernel(PrefArgs p) {
  constexpr int kHalf = kPairWaves / 2;
  __shared__ double part[kPairWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, P = p.S / 2, q = (int)blockIdx.x;
  const int64_t base = (int64_t)(q + (wave / kHalf) * P) * p.T;
  double v = 0.0;
#pragma unroll 4
  for (int i = 64 * (wave % kHalf) + lane; i < p.T; i += 64 * kHalf) {
    const int64_t y = p.labels[base + i];
    const double d = (double)p.lp[base + i] - (double)p.ref[base + i];
    v += y >= 0 && y < p.V ? d : 0.0;
  }
  v = wave_sum(v);
  if (lane == 0) part[wave] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    double sa = part[0], sb = part[kHalf];
    for (int k = 1; k < kHalf; ++k) {
      sa += part[k];
      sb += part[kHalf + k];
    }
    const double ra = (double)p.beta * sa, rb = (double)p.beta * sb, h = ra - rb;
    const double w = -(double)p.gscale * ((double)p.beta / P) * (1.0 / (1.0 + exp(h)) - (double)p.eps);
    p.pair[q] = (1.0 - (double)p.eps) * softplus(-h) + (double)p.eps * softplus(h);
    p.reward[q] = (float)ra;
    p.reward[P + q] = (float)rb;
    p.w[q] = (float)w;
    p.w[P + q] = (float)-w;
  }
}

// The mean of the pairs' losses, by one wave (lane l: pairs l, l + 64, ...).
__device__ __forceinline__ void mean_loss(const PrefArgs& p) {
  const int P = p.S / 2;
  double v = 0.0;
  for (int q = (int)threadIdx.x; q < P; q += 64) v += p.pair[q];
  v = wave_sum(v);
  if (threadIdx.x == 0) *p.loss = P > 0 ? (float)(v / P) : 0.0f;
}

template <typename T>
__global__ __launch_bounds__(kRowThreads) void row_grad_kernel(PrefArgs p) {
  const int tid = threadIdx.x;
  const int64_t row = p.rows - 1 - row_number();
  if (row < 0) {                         // one more workgroup than rows
    if (row == -1 && tid < 64) mean_loss(p);
    return;
  }
  const int64_t y = p.labels[row];
  constexpr int N = Vec<T>::kN;
  T* dx = static_cast<T*>(p.dx) + row * p.ldd;
  if (y < 0 || y >= p.V) {
    const RowParts<T> d(dx, p.V);
    if (tid < d.head) dx[tid] = 0;
    if (tid < p.V - d.tail0) dx[d.tail0 + tid] = 0;
    u32x4_t* dv = reinterpret_cast<u32x4_t*>(dx + d.head);
    for (int i = tid; i < d.pieces; i += kRowThreads) __builtin_nontemporal_store(u32x4_t{0u, 0u, 0u, 0u}, dv + i);
    return;
  }
  const T* x = static_cast<const T*>(p.x) + row * p.ld;
  const f32x2_t st = p.stat[row];
  const float m = st.x, w = p.w[row / p.T], wi = -w * st.y;
  const int yy = (int)y;
  auto one = [&](int v, float xv) {
    const float e = exp_neg(xv - m);
    return v == yy ? w * (1.0f - e * st.y) : wi * e;
  };
  const RowParts<T> r(x, p.V);
  if (((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(dx)) & 15u) == 0) {
    if (tid < r.head) dx[tid] = Vec<T>::round(one(tid, Vec<T>::one(x[tid])));
    if (tid < p.V - r.tail0) dx[r.tail0 + tid] = Vec<T>::round(one(r.tail0 + tid, Vec<T>::one(x[r.tail0 + tid])));
    const u32x4_t* xv = reinterpret_cast<const u32x4_t*>(x + r.head);
    u32x4_t* dv = reinterpret_cast<u32x4_t*>(dx + r.head);
    constexpr int kU = 4;
    for (int b = tid; b < r.pieces; b += kU * kRowThreads) {
      u32x4_t raw[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int i = b + u * kRowThreads;
        raw[u] = xv[i < r.pieces ? i : b];
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int i = b + u * kRowThreads;
        float v[N];
        Vec<T>::unpack(raw[u], v);
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = one(r.head + i * N + e, v[e]);
        if (i < r.pieces) __builtin_nontemporal_store(Vec<T>::pack(v), dv + i);
      }
    }
  } else {  // differently aligned rows (other strides or base offsets): element by element
    for (int v = tid; v < p.V; v += kRowThreads) dx[v] = Vec<T>::round(one(v, Vec<T>::one(x[v])));
  }
}

template <typename T>
hipError_t run_preference(PrefArgs& p, bool grad, hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (p.rows > 0) {
    hipLaunchKernelGGL((row_stats_kernel<T>), row_grid(p.rows), dim3(kRowThreads), 0, stream, p);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (p.S > 0) {
    hipLaunchKernelGGL(pair_loss_kernel, dim3((unsigned)(p.S / 2)), dim3(64 * kPairWaves), 0, stream, p);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (!grad) p.rows = 0;   // only the mean's workgroup
  hipLaunchKernelGGL((row_grad_kernel<T>), row_grid(p.rows + 1), dim3(kRowThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_preference(const PrefCall& c, hipStream_t stream) {
  PrefArgs p;
  p.x = c.logits; p.labels = c.labels; p.ref = c.ref; p.dx = c.dlogits;
  p.lp = c.logps; p.reward = c.rewards; p.loss = c.loss;
  char* ws = static_cast<char*>(c.ws);
  const PrefWorkspace L = pref_workspace_layout(c.S / 2, c.T);
  p.stat = reinterpret_cast<f32x2_t*>(ws + L.stat_off);
  p.pair = reinterpret_cast<double*>(ws + L.pair_off);
  p.w = reinterpret_cast<float*>(ws + L.weight_off);
  p.rows = (int64_t)c.S * c.T;
  p.ld = c.ld; p.ldd = c.ldd;
  p.S = c.S; p.T = c.T; p.V = c.V;
  p.beta = c.beta; p.eps = c.eps; p.gscale = c.gscale;
  const bool grad = c.dlogits != nullptr;
  return c.bf16 ? run_preference<uint16_t>(p, grad, stream) : run_preference<float>(p, grad, stream);
}

}  // namespace qlora
