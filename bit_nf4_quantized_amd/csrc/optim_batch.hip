// The optimiser step over many separately allocated adapter tensors, for
// gfx950: one global gradient norm and one AdamW step per call, with the two
// state vectors held in fp32 or in 8 bits.
//
// The tensors of a call are described by a table in the kernel arguments. A
// tensor is cut into chunks of kChunk values, and a workgroup finds its tensor
// by counting the first-chunk numbers at or below its own, one table entry per
// lane and step. 4 KB of arguments hold 112 tensors of a step or 256 of a norm:
// sizes are kept as the chunk numbers and the values in the last chunk, state
// places in blocks. 448 tensors of 160 M values, clip and 8-bit step: 683 us
// with 4 + 2 launches, 735 us with 64 entries of 8-byte fields and 7 + 7.
//
// State layout (both widths): one array per state vector for all tensors,
// tensor k's values from off_k = sum_{j < k} 256 ceil(n_j / 256), so that a
// block of 256 values never spans two tensors and every access is aligned.
//
// 8-bit state. Per block of 256 values: scale = RN32(top / 448) with top the
// largest magnitude, and an E4M3 code (OCP E4M3FN, nearest, ties to even) of
// RN32(x * RN32(448 / top)) per value; a top below 2^-100 gives zeros. What is
// held is m, and r = sqrt(v) rather than v: Adam divides by sqrt(v), and the
// square root halves the exponent range, so E4M3's 2^-17.8 .. 1 of a block's
// largest value covers gradients that differ by 2^17 within a block (v itself
// would be covered over 2^9 only). The 3 mantissa bits put an error of at
// most 6 % on an element's step. r > 0 never rounds to code 0: a lost r would
// leave eps alone in the denominator, and the next step would be m / eps.
// The step itself uses the unrounded m and v of this step.
//
// Both kernels stream: per value adamw moves theta 8 B, the gradient 4 or 2,
// the bf16 copy 2, and the state 16 B (fp32) or 4 B + 4 / 64 (8 bits); they
// are bound by HBM. A wave owns whole state blocks (4 values per lane, so
// theta and g are 16-byte accesses): the block maximum is one wave reduction,
// with no LDS and no barrier, and the loads of kBlocksPerWave blocks are in
// flight together. The norm reads the tensors forwards and the step goes
// through them backwards, so that it finds the gradients read last in the
// 256 MB memory-side cache; its stores are not read again and are non-temporal
// (692 -> 683 us). Sums are in float64 in a fixed order; no atomics.
//
// That case: adamw_batch_kernel 4 x 152 us (18 B a value, 4.7 TB/s),
// sumsq_batch_kernel 2 x 70 us (4.6 TB/s), clip_finalize_kernel 5 us. 14
// tensors of 0.62 M values in all (fp32 state): 7.1 + 4.5 + 2.3 us of kernels
// in 20 us, which the host's two calls and three launches bound. A maximum
// without LDS exchanges (lane rotations) changed neither (683 / 688 us).
#include "adam.h"
#include "common.h"
#include "launch.h"

namespace qlora {

namespace {

constexpr int kBatchWaves = 4;
constexpr int kBlocksPerWave = 4;
constexpr int kStateBlock = 256;     // 64 lanes x 4 values
constexpr int kChunk = kBatchWaves * kBlocksPerWave * kStateBlock;
constexpr int kStepItems = 112, kNormItems = 256;

// first[k]: chunks of the tensors before k in this launch (first[n] = all);
// unused entries hold INT32_MAX. tail[k]: values in the tensor's last chunk.
template <int ITEMS>
struct BatchHead {
  int32_t first[ITEMS + 1];
  int32_t n;
  uint16_t tail[ITEMS];
};

struct StepTable {
  BatchHead<kStepItems> head;
  float* theta[kStepItems];
  const void* g[kStepItems];
  uint16_t* theta16[kStepItems];
  uint32_t block[kStepItems];        // first state block
};

struct NormTable {
  BatchHead<kNormItems> head;
  const void* g[kNormItems];
};

static_assert(sizeof(StepTable) <= 4000 && sizeof(NormTable) <= 4000, "kernel arguments end at 4 KB");

// The tensor of chunk c of the launch (wave-uniform).
template <int ITEMS>
__device__ __forceinline__ int item_of(const BatchHead<ITEMS>& h, int c) {
  const int lane = threadIdx.x & 63;
  int below = 0;
#pragma unroll
  for (int base = 0; base < ITEMS; base += 64) {
    const int i = base + lane;
    below += __popcll(__ballot(i < ITEMS && h.first[i < ITEMS ? i : 0] <= c));
  }
  return __builtin_amdgcn_readfirstlane(below - 1);
}

template <int ITEMS>
__device__ __forceinline__ int64_t numel_of(const BatchHead<ITEMS>& h, int item) {
  return (int64_t)(h.first[item + 1] - h.first[item] - 1) * kChunk + h.tail[item];
}

// Four values from i on; those at or past n read as 0 (FULL: none are).
template <bool FULL>
__device__ __forceinline__ f32x4_t load4(const float* p, int64_t i, int64_t n) {
  if (FULL || i + 4 <= n) return *reinterpret_cast<const f32x4_t*>(p + i);
  f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int e = 0; e < 3; ++e)
    if (i + e < n) v[e] = p[i + e];
  return v;
}

template <bool FULL>
__device__ __forceinline__ f32x4_t load4(const uint16_t* p, int64_t i, int64_t n) {
  if (FULL || i + 4 <= n) {
    const u32x2_t w = *reinterpret_cast<const u32x2_t*>(p + i);
    return f32x4_t{bf16_to_f32(w.x), bf16_to_f32(w.x >> 16), bf16_to_f32(w.y), bf16_to_f32(w.y >> 16)};
  }
  f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int e = 0; e < 3; ++e)
    if (i + e < n) v[e] = bf16_to_f32(p[i + e]);
  return v;
}

// Four E4M3 codes of a state array; its allocation covers whole blocks.
__device__ __forceinline__ f32x4_t decode4(uint32_t w, float scale) {
  const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  return f32x4_t{lo.x * scale, lo.y * scale, hi.x * scale, hi.y * scale};
}

__device__ __forceinline__ uint32_t encode4(const f32x4_t& x, float inv, bool keep) {
  float y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    y[e] = x[e] * inv;
    if (keep && y[e] > 0.0f) y[e] = __builtin_fmaxf(y[e], 0x1p-9f);
  }
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
  return (uint32_t)w;
}

__device__ __forceinline__ float top4(const f32x4_t& x) {
  const float a = __builtin_fmaxf(__builtin_fabsf(x[0]), __builtin_fabsf(x[1]));
  const float b = __builtin_fmaxf(__builtin_fabsf(x[2]), __builtin_fabsf(x[3]));
  return wave_max(__builtin_fmaxf(a, b), 64);
}

struct StepState {
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
};

template <bool BITS8, typename G, bool FULL>
__device__ __forceinline__ void step_chunk(const StepTable& t, int item, int64_t base, const StepState& st,
                                           const AdamConsts& k, float cf) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n = numel_of(t.head, item), off = (int64_t)t.block[item] * kStateBlock;
  float* theta = t.theta[item];
  const G* g = static_cast<const G*>(t.g[item]);
  uint16_t* theta16 = t.theta16[item];
  f32x4_t th[kBlocksPerWave], gr[kBlocksPerWave], m[kBlocksPerWave], v[kBlocksPerWave];
  uint32_t mc[kBlocksPerWave], vc[kBlocksPerWave];
  float ms[kBlocksPerWave], vs[kBlocksPerWave];
  auto start = [&](int b) { return base + (int64_t)(wave + kBatchWaves * b) * kStateBlock; };  // first value of the block
#pragma unroll
  for (int b = 0; b < kBlocksPerWave; ++b) {
    const int64_t s0 = start(b), i = s0 + 4 * lane;
    if (!FULL && s0 >= n) continue;
    th[b] = load4<FULL>(theta, i, n);
    gr[b] = load4<FULL>(g, i, n);
    if constexpr (BITS8) {
      mc[b] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(st.m) + off + i);
      vc[b] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(st.v) + off + i);
      ms[b] = st.m_scale[(off + s0) / kStateBlock];
      vs[b] = st.v_scale[(off + s0) / kStateBlock];
    } else {
      m[b] = *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(st.m) + off + i);
      v[b] = *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(st.v) + off + i);
    }
  }
#pragma unroll
  for (int b = 0; b < kBlocksPerWave; ++b) {
    const int64_t s0 = start(b), i = s0 + 4 * lane;
    if (!FULL && s0 >= n) continue;
    if constexpr (BITS8) {
      m[b] = decode4(mc[b], ms[b]);
      const f32x4_t r = decode4(vc[b], vs[b]);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[b][e] = r[e] * r[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a = th[b][e], mm = m[b][e], vv = v[b][e];
      adam_one(a, gr[b][e], mm, vv, cf, k);
      th[b][e] = a;
      m[b][e] = mm;
      v[b][e] = vv;
      if (!FULL && i + e >= n) m[b][e] = v[b][e] = 0.0f;   // the padding of a last block stays 0
    }
    if (FULL || i + 4 <= n) {
      __builtin_nontemporal_store(th[b], reinterpret_cast<f32x4_t*>(theta + i));
      if (theta16)
        __builtin_nontemporal_store((u32x2_t{pack_bf16x2(th[b][0], th[b][1]), pack_bf16x2(th[b][2], th[b][3])}), reinterpret_cast<u32x2_t*>(theta16 + i));
    } else {
      for (int e = 0; e < 3; ++e)
        if (i + e < n) {
          theta[i + e] = th[b][e];
          if (theta16) theta16[i + e] = f32_to_bf16(th[b][e]);
        }
    }
    if constexpr (BITS8) {
      f32x4_t r;
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = __builtin_sqrtf(v[b][e]);
      const float mt = top4(m[b]), rt = top4(r);
      const bool mz = mt < 0x1p-100f, rz = rt < 0x1p-100f;
      const uint32_t mq = encode4(m[b], mz ? 0.0f : 448.0f / mt, false);
      const uint32_t rq = encode4(r, rz ? 0.0f : 448.0f / rt, true);
      __builtin_nontemporal_store(mq, reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(st.m) + off + i));
      __builtin_nontemporal_store(rq, reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(st.v) + off + i));
      if (lane == 0) {
        st.m_scale[(off + s0) / kStateBlock] = mz ? 0.0f : mt / 448.0f;
        st.v_scale[(off + s0) / kStateBlock] = rz ? 0.0f : rt / 448.0f;
      }
    } else {
      __builtin_nontemporal_store(m[b], reinterpret_cast<f32x4_t*>(static_cast<float*>(st.m) + off + i));
      __builtin_nontemporal_store(v[b], reinterpret_cast<f32x4_t*>(static_cast<float*>(st.v) + off + i));
    }
  }
}

template <bool BITS8, typename G>
__global__ __launch_bounds__(64 * kBatchWaves) void adamw_batch_kernel(StepTable t, StepState st, AdamConsts k,
                                                                       const float* __restrict__ coef) {
  const int item = item_of(t.head, (int)blockIdx.x);
  const int64_t base = (int64_t)(t.head.first[item + 1] - 1 - (int)blockIdx.x) * kChunk;
  const float cf = coef ? *coef : 1.0f;
  if (base + kChunk <= numel_of(t.head, item))
    step_chunk<BITS8, G, true>(t, item, base, st, k, cf);
  else
    step_chunk<BITS8, G, false>(t, item, base, st, k, cf);
}

// part[b] (+)= the squares of chunks b, b + gridDim, ... of this launch.
template <typename G>
__global__ __launch_bounds__(256) void sumsq_batch_kernel(NormTable t, int add, double* __restrict__ part) {
  __shared__ double s[256];
  const int total = t.head.first[t.head.n];
  double acc = 0.0;
  for (int c = (int)blockIdx.x; c < total; c += kNormBlocks) {
    const int item = item_of(t.head, c);
    const int64_t n = numel_of(t.head, item);
    const int64_t base = (int64_t)(c - t.head.first[item]) * kChunk + 4 * (int)threadIdx.x;
    const G* g = static_cast<const G*>(t.g[item]);
    f32x4_t x[kChunk / 1024];
#pragma unroll
    for (int u = 0; u < kChunk / 1024; ++u) x[u] = load4<false>(g, base + 1024 * u, n);
#pragma unroll
    for (int u = 0; u < kChunk / 1024; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc += (double)x[u][e] * x[u][e];
  }
  const double tot = tree_sum_256(acc, s);
  if (threadIdx.x == 0) part[blockIdx.x] = add ? part[blockIdx.x] + tot : tot;
}

// Fills the table with tensors at, at + step, ... (step 1 or -1), as far as
// entries and 31-bit chunk numbers go; returns the first one not taken.
// take(slot, k) copies tensor k's fields.
template <int ITEMS, typename Take>
int fill_table(BatchHead<ITEMS>& h, int at, int step, int n, const int64_t* numel, Take&& take) {
  for (int i = 0; i <= ITEMS; ++i) h.first[i] = 0x7FFFFFFF;
  int used = 0;
  int64_t chunks = 0;
  for (; at >= 0 && at < n && used < ITEMS; at += step) {
    if (numel[at] == 0) continue;
    const int64_t c = (numel[at] + kChunk - 1) / kChunk;
    if (used > 0 && chunks + c > 0x7FFFFFFE) break;
    h.first[used] = (int32_t)chunks;
    h.tail[used] = (uint16_t)(numel[at] - (c - 1) * kChunk);
    take(used++, at);
    chunks += c;
  }
  h.n = used;
  h.first[used] = (int32_t)chunks;   // the launch's chunks; above every chunk number
  return at;
}

}  // namespace

hipError_t launch_clip_norm_batch(int n, const void* const* g, bool g16, const int64_t* numel, double max_norm,
                                  float* coef, double* norm, double* part, hipStream_t stream) {
  int at = 0, add = 0;
  do {
    NormTable t;
    at = fill_table(t.head, at, 1, n, numel, [&](int slot, int k) {
      t.g[slot] = g[k];
    });
    if (g16)
      hipLaunchKernelGGL(sumsq_batch_kernel<uint16_t>, dim3(kNormBlocks), dim3(256), 0, stream, t, add, part);
    else
      hipLaunchKernelGGL(sumsq_batch_kernel<float>, dim3(kNormBlocks), dim3(256), 0, stream, t, add, part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    add = 1;
  } while (at < n);
  hipLaunchKernelGGL(clip_finalize_kernel, dim3(1), dim3(1024), 0, stream, part, max_norm, coef, norm);
  return hipGetLastError();
}

hipError_t launch_adamw_batch(const AdamBatch& b, const AdamHyper& h, const float* coef, hipStream_t stream) {
  const AdamConsts kc = adam_consts(h);
  const StepState st{b.m, b.v, b.m_scale, b.v_scale};
  int64_t off = 0;    // where the state of tensor `seen` begins
  int seen = b.n;
  for (int k = 0; k < b.n; ++k) off += adam_state_span(b.numel[k]);
  for (int at = b.n - 1; at >= 0;) {
    StepTable t;
    at = fill_table(t.head, at, -1, b.n, b.numel, [&](int slot, int i) {
      while (seen > i) off -= adam_state_span(b.numel[--seen]);
      t.theta[slot] = b.theta[i];
      t.g[slot] = b.g[i];
      t.theta16[slot] = b.theta16 ? b.theta16[i] : nullptr;
      t.block[slot] = (uint32_t)(off / kStateBlock);
    });
    if (t.head.n == 0) break;
    const dim3 grid((unsigned)t.head.first[t.head.n]), block(64 * kBatchWaves);
    if (b.bits8 && b.g16)
      hipLaunchKernelGGL((adamw_batch_kernel<true, uint16_t>), grid, block, 0, stream, t, st, kc, coef);
    else if (b.bits8)
      hipLaunchKernelGGL((adamw_batch_kernel<true, float>), grid, block, 0, stream, t, st, kc, coef);
    else if (b.g16)
      hipLaunchKernelGGL((adamw_batch_kernel<false, uint16_t>), grid, block, 0, stream, t, st, kc, coef);
    else
      hipLaunchKernelGGL((adamw_batch_kernel<false, float>), grid, block, 0, stream, t, st, kc, coef);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace qlora
