// C ABI of the QLoRA NF4 library: host-side validation, sizes, the NF4
// codebook, and stream-ordered kernel launches. See include/qlora_nf4.h,
// include/qlora_adapters.h and include/qlora_layers.h.
#include "qlora_adapters.h"
#include "qlora_layers.h"
#include "qlora_nf4.h"

#include <math.h>
#include <stdio.h>
#include <string.h>

#include <mutex>

#include "launch.h"

using qlora::LinearWorkspace;
using qlora::NF4Table;
using qlora::NF4Thresholds;
using qlora::NF4View;

namespace {

thread_local char g_last_error[256] = "";

int hip_fail(hipError_t e) {
  snprintf(g_last_error, sizeof(g_last_error), "%s: %s", hipGetErrorName(e), hipGetErrorString(e));
  return QLORA_ERR_HIP;
}

static_assert(qlora::kMultiMaxRows == QLORA_MULTI_MAX_ROWS && qlora::kMultiMaxAdapters == QLORA_MULTI_MAX_ADAPTERS,
              "limits of the header and of the kernels");
static_assert(qlora::kLayerMaxRows == QLORA_LAYER_MAX_ROWS && qlora::kNormMaxK == QLORA_NORM_MAX_COLS &&
                  qlora::kHeadMaxVocab == QLORA_HEAD_MAX_VOCAB && qlora::kGatedMaxCols == QLORA_GATED_MAX_COLS,
              "limits of the header and of the kernels");

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// N(0,1) quantile by bisection on the CDF 1/2 erfc(-x / sqrt 2), to full
// double precision.
double normal_quantile(double p) {
  double lo = -40.0, hi = 40.0;
  for (int i = 0; i < 400; ++i) {
    const double mid = 0.5 * (lo + hi);
    if (mid == lo || mid == hi) break;
    if (0.5 * erfc(-mid / sqrt(2.0)) < p)
      lo = mid;
    else
      hi = mid;
  }
  return 0.5 * (lo + hi);
}

// S_c = { 1/2 [Q(i/(c+2)) + Q((i+1)/(c+2))] : i = 1..c } for odd c (QLoRA
// pages, diycv.top, section 方法总览 item 2, with c = 15 giving the
// denominator 2^4 + 1); its middle element is exactly 0.
void quantile_set(int c, double* out) {
  const double d = (double)(c + 2);
  for (int i = 1; i <= c; ++i) out[i - 1] = 0.5 * (normal_quantile(i / d) + normal_quantile((i + 1) / d));
  out[c / 2] = 0.0;
}

struct Tables {
  NF4Table tab;
  NF4Thresholds th;
};

// The 16 ascending table values of a 4-bit data type, in float64 before the
// one fp32 rounding.
//   NF4: 7 negative members of S_15 over |min S_15|, an exact 0, and 8
//     positive members of S_17 over max S_17 (diycv.top, section 方法总览
//     item 2).
//   Int4: the Int8 absmax formula of the same section (item 1) with 4-bit
//     signed integers, levels k/7; entry k + 8 holds k/7 for k = -8..7
//     (k = -8 is never produced: |x| <= 1).
//   FP4 E2M1 (1 sign, 2 exponent bits with bias 1, 1 mantissa bit: 0, 0.5,
//     1, 1.5, 2, 3, 4, 6) and FP4 E3M0 (exponent field 0 = zero, else a
//     power of two: 0, 2^-6 .. 1 after scaling) scaled so that the largest
//     magnitude is 1; +-0 are one value, so entry 0 holds an unused -2.
//   (The pages name Int4, FP4 E2M1 and FP4 E3M0 in section 实验设置与主要结果
//   item 1 without defining them; these are the plainest readings.)
void type_values(int qtype, double* v) {
  if (qtype == QLORA_QTYPE_NF4) {
    double s15[15], s17[17];
    quantile_set(15, s15);
    quantile_set(17, s17);
    int n = 0;
    for (int i = 0; i < 7; ++i) v[n++] = s15[i] / (-s15[0]);
    v[n++] = 0.0;
    for (int i = 9; i < 17; ++i) v[n++] = s17[i] / s17[16];
    v[0] = -1.0;
    v[15] = 1.0;
  } else if (qtype == QLORA_QTYPE_INT4) {
    for (int k = -8; k < 8; ++k) v[k + 8] = (double)k / 7.0;
  } else {
    const double e2m1[7] = {0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0};
    double mag[7];
    for (int i = 0; i < 7; ++i) mag[i] = qtype == QLORA_QTYPE_FP4_E2M1 ? e2m1[i] / 6.0 : ldexp(1.0, i - 6);
    v[0] = -2.0;
    for (int i = 0; i < 7; ++i) v[1 + i] = -mag[6 - i];
    v[8] = 0.0;
    for (int i = 0; i < 7; ++i) v[9 + i] = mag[i];
  }
}

// The table of a data type (one fp32 rounding per value), plus the decision
// thresholds between neighbouring codes.
Tables build_tables(int qtype) {
  double v[16];
  type_values(qtype, v);
  Tables T;
  for (int i = 0; i < 16; ++i) T.tab.q[i] = (float)v[i];
  for (int j = 0; j < 15; ++j) {
    // exact midpoint of two fp32 values, then the smallest fp32 strictly above it
    const double m = 0.5 * ((double)T.tab.q[j] + (double)T.tab.q[j + 1]);
    float f = (float)m;
    if (!((double)f > m)) f = nextafterf(f, INFINITY);
    T.th.t[j] = f;
  }
  return T;
}

constexpr int kQTypes = 4;

const Tables& tables(int qtype) {
  static const Tables T[kQTypes] = {build_tables(0), build_tables(1), build_tables(2), build_tables(3)};  // one-time init
  return T[qtype];
}

bool valid_qtype(int qtype) { return qtype >= 0 && qtype < kQTypes; }

bool valid_nf4(const qlora_nf4* q) {
  if (!q || !q->codes || !valid_qtype(q->qtype) || (q->no_dq != 0 && q->no_dq != 1)) return false;
  return q->no_dq ? q->absmax32 != nullptr : (q->absmax8 && q->scale2 && q->mean);
}

NF4View view_of(const qlora_nf4* q) {
  NF4View v;
  v.codes = q->codes;
  v.absmax8 = q->absmax8;
  v.scale2 = q->scale2;
  v.mean = q->mean;
  v.rows = q->rows;
  v.cols = q->cols;
  v.absmax32 = q->no_dq ? q->absmax32 : nullptr;
  return v;
}

// Shape rules shared by the linear entry points.
int check_linear(const qlora_nf4* W, int64_t M, int r, float scale) {
  if (!valid_nf4(W)) return QLORA_ERR_ARG;
  if (!isfinite(scale)) return QLORA_ERR_ARG;
  if (r < 8 || r > QLORA_MAX_RANK || (r % 8) != 0) return QLORA_ERR_ARG;
  if (M < 0 || W->rows <= 0 || W->cols <= 0) return QLORA_ERR_SHAPE;
  if ((W->cols % QLORA_BLOCK) != 0 || (W->rows % 8) != 0) return QLORA_ERR_SHAPE;
  if (M > (int64_t)1 << 31 || W->rows > (int64_t)1 << 31 || W->cols > (int64_t)1 << 31) return QLORA_ERR_SHAPE;
  if (!aligned16(W->codes)) return QLORA_ERR_ALIGN;
  return QLORA_OK;
}

// log2 of an Int8 codec block size (a power of two in [64, 4096]), or -1.
int int8_block_log2(int block) {
  for (int lg = 6; lg <= 12; ++lg)
    if (block == (1 << lg)) return lg;
  return -1;
}

}  // namespace

extern "C" {

const char* qlora_status_str(int status) {
  switch (status) {
    case QLORA_OK: return "QLORA_OK";
    case QLORA_ERR_ARG: return "QLORA_ERR_ARG: invalid argument";
    case QLORA_ERR_SHAPE: return "QLORA_ERR_SHAPE: unsupported or inconsistent shape";
    case QLORA_ERR_ALIGN: return "QLORA_ERR_ALIGN: device pointer not 16-byte aligned";
    case QLORA_ERR_WORKSPACE: return "QLORA_ERR_WORKSPACE: workspace missing or too small";
    case QLORA_ERR_HIP: return "QLORA_ERR_HIP: HIP runtime or launch failure";
    default: return "unknown qlora status";
  }
}

const char* qlora_last_error(void) { return g_last_error; }

int qlora_nf4_codebook(float* out16) {
  if (!out16) return QLORA_ERR_ARG;
  memcpy(out16, tables(QLORA_QTYPE_NF4).tab.q, sizeof(float) * 16);
  return QLORA_OK;
}

int qlora_codebook(int qtype, float* out16) {
  if (!out16 || !valid_qtype(qtype)) return QLORA_ERR_ARG;
  memcpy(out16, tables(qtype).tab.q, sizeof(float) * 16);
  return QLORA_OK;
}

int qlora_quant_sizes(int64_t rows, int64_t cols, size_t* codes_bytes, size_t* absmax8_bytes,
                      size_t* scale2_bytes, size_t* workspace_bytes) {
  if (rows < 0 || cols < 0) return QLORA_ERR_SHAPE;
  if (cols > 0 && rows > INT64_MAX / 2 / cols) return QLORA_ERR_SHAPE;
  const int64_t numel = rows * cols;
  const int64_t nb = (numel + QLORA_BLOCK - 1) / QLORA_BLOCK;
  const int64_t ng = (nb + QLORA_DQ_BLOCK - 1) / QLORA_DQ_BLOCK;
  if (codes_bytes) *codes_bytes = (size_t)((numel + 1) / 2);
  if (absmax8_bytes) *absmax8_bytes = (size_t)nb;
  if (scale2_bytes) *scale2_bytes = (size_t)ng * sizeof(float);
  if (workspace_bytes) *workspace_bytes = qlora::quant_workspace_layout(numel).total;
  return QLORA_OK;
}

int qlora_quantize(const void* W, qlora_dtype in_dtype, const qlora_nf4* q, void* ws, size_t ws_bytes,
                   hipStream_t stream) {
  if (!q) return QLORA_ERR_ARG;
  if (in_dtype != QLORA_F32 && in_dtype != QLORA_BF16) return QLORA_ERR_ARG;
  if (q->rows < 0 || q->cols < 0) return QLORA_ERR_SHAPE;
  if (q->cols > 0 && q->rows > INT64_MAX / 2 / q->cols) return QLORA_ERR_SHAPE;
  const int64_t numel = q->rows * q->cols;
  if (numel == 0) return QLORA_OK;
  if ((numel + QLORA_BLOCK * QLORA_DQ_BLOCK - 1) / (QLORA_BLOCK * QLORA_DQ_BLOCK) > 0x7FFFFFFF)
    return QLORA_ERR_SHAPE;
  if (!W || !valid_nf4(q) || !ws) return QLORA_ERR_ARG;
  if (!aligned16(W) || !aligned16(q->codes) || !aligned16(ws)) return QLORA_ERR_ALIGN;
  if (ws_bytes < qlora::quant_workspace_layout(numel).total) return QLORA_ERR_WORKSPACE;
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e = qlora::launch_quantize(W, in_dtype == QLORA_BF16, numel, tables(q->qtype).th, q->codes,
                                              q->absmax8, q->scale2, q->mean, q->no_dq ? q->absmax32 : nullptr,
                                              ws, stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

// Byte offset of tensor k's scratch in a batch workspace (each part rounded
// up to 256); k = n gives the total.
static size_t batch_ws_offset(int k, const int64_t* numel) {
  size_t off = 0;
  for (int j = 0; j < k; ++j) off += qlora::align_up(qlora::quant_workspace_layout(numel[j]).total, 256);
  return off;
}

// rows/cols -> numel with the single-tensor shape rules; QLORA_OK or an error.
static int batch_numel(int64_t rows, int64_t cols, int64_t* numel) {
  if (rows < 0 || cols < 0) return QLORA_ERR_SHAPE;
  if (cols > 0 && rows > INT64_MAX / 2 / cols) return QLORA_ERR_SHAPE;
  *numel = rows * cols;
  if ((*numel + QLORA_BLOCK * QLORA_DQ_BLOCK - 1) / (QLORA_BLOCK * QLORA_DQ_BLOCK) > 0x7FFFFFFF)
    return QLORA_ERR_SHAPE;
  return QLORA_OK;
}

int qlora_quant_batch_workspace(int n, const int64_t* rows, const int64_t* cols, size_t* bytes) {
  if (n < 1 || n > QLORA_QUANT_BATCH_MAX || !rows || !cols || !bytes) return QLORA_ERR_ARG;
  int64_t numel[QLORA_QUANT_BATCH_MAX];
  for (int k = 0; k < n; ++k) {
    const int st = batch_numel(rows[k], cols[k], &numel[k]);
    if (st != QLORA_OK) return st;
  }
  *bytes = batch_ws_offset(n, numel);
  return QLORA_OK;
}

int qlora_quantize_batch(int n, const void* const* W, qlora_dtype in_dtype, const qlora_nf4* const* q, void* ws,
                         size_t ws_bytes, hipStream_t stream) {
  if (n < 1 || n > QLORA_QUANT_BATCH_MAX || !W || !q) return QLORA_ERR_ARG;
  if (in_dtype != QLORA_F32 && in_dtype != QLORA_BF16) return QLORA_ERR_ARG;
  int64_t numel[QLORA_QUANT_BATCH_MAX];
  int first = -1;                                // the first non-empty tensor
  for (int k = 0; k < n; ++k) {
    if (!q[k]) return QLORA_ERR_ARG;
    const int st = batch_numel(q[k]->rows, q[k]->cols, &numel[k]);
    if (st != QLORA_OK) return st;
    if (numel[k] == 0) continue;
    if (!W[k] || !valid_nf4(q[k])) return QLORA_ERR_ARG;
    if (first < 0) first = k;
    if (q[k]->qtype != q[first]->qtype) return QLORA_ERR_ARG;     // one threshold table per launch
    if (!aligned16(W[k]) || !aligned16(q[k]->codes)) return QLORA_ERR_ALIGN;
  }
  if (first < 0) return QLORA_OK;                // nothing to quantise
  int64_t groups = 0;                            // one workgroup per DQ group of the whole batch
  for (int k = 0; k < n; ++k) groups += (numel[k] + QLORA_BLOCK * QLORA_DQ_BLOCK - 1) / (QLORA_BLOCK * QLORA_DQ_BLOCK);
  if (groups > 0x7FFFFFFF) return QLORA_ERR_SHAPE;
  if (!ws) return QLORA_ERR_ARG;
  if (!aligned16(ws)) return QLORA_ERR_ALIGN;
  if (ws_bytes < batch_ws_offset(n, numel)) return QLORA_ERR_WORKSPACE;
  qlora::QuantItem items[QLORA_QUANT_BATCH_MAX];
  for (int k = 0; k < n; ++k) {
    const qlora_nf4* t = q[k];
    items[k] = qlora::QuantItem{W[k], numel[k], t->codes, t->absmax8, t->scale2, t->mean,
                                t->no_dq ? t->absmax32 : nullptr, static_cast<char*>(ws) + batch_ws_offset(k, numel)};
  }
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e =
      qlora::launch_quantize_batch(items, n, in_dtype == QLORA_BF16, tables(q[first]->qtype).th, stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

int qlora_dequantize(const qlora_nf4* q, uint16_t* out, hipStream_t stream) {
  if (!q) return QLORA_ERR_ARG;
  if (q->rows < 0 || q->cols < 0) return QLORA_ERR_SHAPE;
  if (q->cols > 0 && q->rows > INT64_MAX / 2 / q->cols) return QLORA_ERR_SHAPE;
  const int64_t numel = q->rows * q->cols;
  if (numel == 0) return QLORA_OK;
  if (!valid_nf4(q) || !out) return QLORA_ERR_ARG;
  if (!aligned16(q->codes) || !aligned16(out)) return QLORA_ERR_ALIGN;
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e =
      qlora::launch_dequantize(q->codes, q->absmax8, q->scale2, q->mean, q->no_dq ? q->absmax32 : nullptr,
                               tables(q->qtype).tab, numel, out, stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

int qlora_int8_quantize(const void* X, qlora_dtype in_dtype, int64_t numel, int block, int8_t* codes,
                        float* absmax, hipStream_t stream) {
  const int lg = int8_block_log2(block);
  if (lg < 0 || (in_dtype != QLORA_F32 && in_dtype != QLORA_BF16)) return QLORA_ERR_ARG;
  if (numel < 0 || numel > QLORA_INT8_MAX_NUMEL) return QLORA_ERR_SHAPE;
  if (numel == 0) return QLORA_OK;
  if (!X || !codes || !absmax) return QLORA_ERR_ARG;
  if (!aligned16(X) || !aligned16(codes) || (reinterpret_cast<uintptr_t>(absmax) & 3u)) return QLORA_ERR_ALIGN;
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e = qlora::launch_int8_quantize(X, in_dtype == QLORA_BF16, numel, lg, codes, absmax, stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

int qlora_int8_dequantize(const int8_t* codes, const float* absmax, int64_t numel, int block, void* out,
                          qlora_dtype out_dtype, hipStream_t stream) {
  const int lg = int8_block_log2(block);
  if (lg < 0 || (out_dtype != QLORA_F32 && out_dtype != QLORA_BF16)) return QLORA_ERR_ARG;
  if (numel < 0 || numel > QLORA_INT8_MAX_NUMEL) return QLORA_ERR_SHAPE;
  if (numel == 0) return QLORA_OK;
  if (!codes || !absmax || !out) return QLORA_ERR_ARG;
  if (!aligned16(codes) || !aligned16(out) || (reinterpret_cast<uintptr_t>(absmax) & 3u)) return QLORA_ERR_ALIGN;
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e =
      qlora::launch_int8_dequantize(codes, absmax, numel, lg, out, out_dtype == QLORA_BF16, stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

int qlora_merge_adapters(const qlora_nf4* W, const uint16_t* L1, const uint16_t* L2, int r, float scale,
                         uint16_t* out, hipStream_t stream) {
  const int st = check_linear(W, 0, r, scale);
  if (st != QLORA_OK) return st;
  if (!L1 || !L2 || !out) return QLORA_ERR_ARG;
  if (!aligned16(L1) || !aligned16(L2) || !aligned16(out)) return QLORA_ERR_ALIGN;
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e = qlora::launch_merge(view_of(W), tables(W->qtype).tab, L1, L2, r, scale, out, stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

int qlora_linear_workspace(int64_t M, int64_t K, int64_t N, int r, size_t* bytes) {
  if (!bytes) return QLORA_ERR_ARG;
  if (r < 8 || r > QLORA_MAX_RANK || (r % 8) != 0) return QLORA_ERR_ARG;
  if (M < 0 || K <= 0 || N <= 0 || (K % QLORA_BLOCK) != 0 || (N % 8) != 0) return QLORA_ERR_SHAPE;
  if (M > (int64_t)1 << 31 || N > (int64_t)1 << 31 || K > (int64_t)1 << 31) return QLORA_ERR_SHAPE;
  *bytes = qlora::linear_workspace_layout(M, K, N, r).total;
  return QLORA_OK;
}

int qlora_linear_workspace_dropout(int64_t M, int64_t K, int64_t N, int r, size_t* bytes) {
  const int st = qlora_linear_workspace(M, K, N, r, bytes);
  if (st != QLORA_OK) return st;
  *bytes = qlora::linear_workspace_layout(M, K, N, r, true).total;
  return QLORA_OK;
}

}  // extern "C"

namespace {

int linear_fwd_impl(const qlora_nf4* W, const uint16_t* X, int64_t M, const uint16_t* L1, const uint16_t* L2, int r,
                    float scale, uint16_t* Y, uint16_t* T_out, void* ws, size_t ws_bytes, hipStream_t stream,
                    const qlora::DropoutParams* dr) {
  int st = check_linear(W, M, r, scale);
  if (st != QLORA_OK) return st;
  if (!L1 || !L2) return QLORA_ERR_ARG;
  if (M > 0 && (!X || !Y)) return QLORA_ERR_ARG;
  if (!ws) return QLORA_ERR_WORKSPACE;
  if (!aligned16(X) || !aligned16(L1) || !aligned16(L2) || !aligned16(Y) || !aligned16(T_out) || !aligned16(ws))
    return QLORA_ERR_ALIGN;
  if (!qlora::linear_forward_supported(M, W->cols, W->rows, r)) return QLORA_ERR_SHAPE;
  if (ws_bytes < qlora::linear_workspace_layout(M, W->cols, W->rows, r, dr != nullptr).total)
    return QLORA_ERR_WORKSPACE;
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e = qlora::linear_forward(view_of(W), tables(W->qtype).tab, X, M, L1, L2, r, scale, Y, T_out, ws,
                                             stream, dr);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

int linear_bwd_impl(const qlora_nf4* W, const uint16_t* X, const uint16_t* dY, int64_t M, const uint16_t* L1,
                    const uint16_t* L2, int r, float scale, const uint16_t* T, uint16_t* dX, void* dL1, void* dL2,
                    qlora_dtype grad_dtype, void* ws, size_t ws_bytes, hipStream_t stream,
                    const qlora::DropoutParams* dr) {
  int st = check_linear(W, M, r, scale);
  if (st != QLORA_OK) return st;
  if (grad_dtype != QLORA_F32 && grad_dtype != QLORA_BF16) return QLORA_ERR_ARG;
  if (!L1 || !L2 || !dL1 || !dL2) return QLORA_ERR_ARG;
  if (M > 0 && (!X || !dY)) return QLORA_ERR_ARG;
  if (!ws) return QLORA_ERR_WORKSPACE;
  if (!aligned16(X) || !aligned16(dY) || !aligned16(L1) || !aligned16(L2) || !aligned16(T) || !aligned16(dX) ||
      !aligned16(dL1) || !aligned16(dL2) || !aligned16(ws))
    return QLORA_ERR_ALIGN;
  if (ws_bytes < qlora::linear_workspace_layout(M, W->cols, W->rows, r, dr != nullptr).total)
    return QLORA_ERR_WORKSPACE;
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e = qlora::linear_backward(view_of(W), tables(W->qtype).tab, X, dY, M, L1, L2, r, scale, T, dX, dL1,
                                              dL2, grad_dtype == QLORA_BF16, ws, stream, dr);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

bool valid_dropout(float p) { return isfinite(p) && p >= 0.0f && p < 1.0f; }

constexpr int64_t kMaxNumel = (int64_t)1 << 40;

bool valid_adam(const qlora_adam_params* hp) {
  return hp && hp->step >= 1 && hp->lr >= 0.0f && isfinite(hp->lr) && hp->eps >= 0.0f && isfinite(hp->eps) &&
         hp->beta1 >= 0.0f && hp->beta1 < 1.0f && hp->beta2 >= 0.0f && hp->beta2 < 1.0f && isfinite(hp->weight_decay);
}

qlora::AdamHyper adam_hyper(const qlora_adam_params* hp) {
  qlora::AdamHyper h;
  h.lr = hp->lr; h.beta1 = hp->beta1; h.beta2 = hp->beta2; h.eps = hp->eps; h.wd = hp->weight_decay;
  h.step = hp->step;
  return h;
}

// The device-side address of p: device memory as it is, pinned host memory
// through its device mapping; nullptr for anything else (pageable host
// memory, managed memory, or an address HIP does not know).
void* device_view(const void* p) {
  hipPointerAttribute_t a;
  if (hipPointerGetAttributes(&a, p) != hipSuccess) {
    (void)hipGetLastError();
    return nullptr;
  }
  if (a.type == hipMemoryTypeDevice && !a.isManaged) return const_cast<void*>(p);
  if (a.type == hipMemoryTypeHost && a.devicePointer && a.hostPointer && !a.isManaged)
    return static_cast<char*>(a.devicePointer) + (static_cast<const char*>(p) - static_cast<const char*>(a.hostPointer));
  return nullptr;
}

// ---- the allocation-free decode forward ----------------------------------------
//
// Scratch of qlora_linear_fwd_noalloc: one array per device, in the module's
// device memory (zero-initialised when the code object loads; held until the
// process ends). Host code never passes the array's name to a kernel: the
// name is a host-side stand-in. The device address comes from
// hipGetSymbolAddress, taken once per device with that device current, and
// that address is what the kernels receive. Calls that overlap on one device
// share the array and race.
__device__ __align__(256) unsigned char scratch[QLORA_NOALLOC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;
void* g_scratch_ptr[kMaxDevices];
std::mutex g_scratch_mu;

// The current device's address of `scratch` (looked up on the first call on
// that device).
int device_scratch(void** out) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e);
  if (dev < 0 || dev >= kMaxDevices) return QLORA_ERR_ARG;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return hip_fail(e);
    if (!p) return hip_fail(hipErrorInvalidSymbol);
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return QLORA_OK;
}

}  // namespace

extern "C" {

int qlora_linear_fwd_noalloc(const qlora_nf4* W, const uint16_t* X, int64_t M, const uint16_t* L1,
                             const uint16_t* L2, int r, float scale, uint16_t* Y, uint16_t* T_out,
                             hipStream_t stream) {
  int st = check_linear(W, M, r, scale);
  if (st != QLORA_OK) return st;
  if (M > 16) return QLORA_ERR_SHAPE;
  if (!L1 || !L2) return QLORA_ERR_ARG;
  if (M > 0 && (!X || !Y)) return QLORA_ERR_ARG;
  if (!aligned16(X) || !aligned16(L1) || !aligned16(L2) || !aligned16(Y) || !aligned16(T_out))
    return QLORA_ERR_ALIGN;
  const qlora::SmallForwardScratch S = qlora::small_forward_scratch(M, W->cols, r);
  if (S.total > QLORA_NOALLOC_SCRATCH_BYTES) return QLORA_ERR_WORKSPACE;
  if (M == 0) return QLORA_OK;
  void* base = nullptr;
  st = device_scratch(&base);
  if (st != QLORA_OK) return st;
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  char* p = static_cast<char*>(base);
  const hipError_t e = qlora::linear_forward_small(
      view_of(W), tables(W->qtype).tab, X, X, M, L1, L2, r, scale, Y, T_out, reinterpret_cast<uint16_t*>(p + S.st_off),
      reinterpret_cast<float*>(p + S.part_off), stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

int qlora_linear_fwd(const qlora_nf4* W, const uint16_t* X, int64_t M, const uint16_t* L1, const uint16_t* L2,
                     int r, float scale, uint16_t* Y, uint16_t* T_out, void* ws, size_t ws_bytes,
                     hipStream_t stream) {
  return linear_fwd_impl(W, X, M, L1, L2, r, scale, Y, T_out, ws, ws_bytes, stream, nullptr);
}

int qlora_linear_bwd(const qlora_nf4* W, const uint16_t* X, const uint16_t* dY, int64_t M, const uint16_t* L1,
                     const uint16_t* L2, int r, float scale, const uint16_t* T, uint16_t* dX, void* dL1,
                     void* dL2, qlora_dtype grad_dtype, void* ws, size_t ws_bytes, hipStream_t stream) {
  return linear_bwd_impl(W, X, dY, M, L1, L2, r, scale, T, dX, dL1, dL2, grad_dtype, ws, ws_bytes, stream, nullptr);
}

int qlora_linear_fwd_dropout(const qlora_nf4* W, const uint16_t* X, int64_t M, const uint16_t* L1,
                             const uint16_t* L2, int r, float scale, float p, uint64_t seed, uint16_t* Y,
                             uint16_t* T_out, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!valid_dropout(p)) return QLORA_ERR_ARG;
  const qlora::DropoutParams d = qlora::dropout_params(p, seed);
  return linear_fwd_impl(W, X, M, L1, L2, r, scale, Y, T_out, ws, ws_bytes, stream, &d);
}

int qlora_linear_bwd_dropout(const qlora_nf4* W, const uint16_t* X, const uint16_t* dY, int64_t M,
                             const uint16_t* L1, const uint16_t* L2, int r, float scale, float p, uint64_t seed,
                             const uint16_t* T, uint16_t* dX, void* dL1, void* dL2, qlora_dtype grad_dtype,
                             void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!valid_dropout(p)) return QLORA_ERR_ARG;
  const qlora::DropoutParams d = qlora::dropout_params(p, seed);
  return linear_bwd_impl(W, X, dY, M, L1, L2, r, scale, T, dX, dL1, dL2, grad_dtype, ws, ws_bytes, stream, &d);
}

int qlora_clip_grad_norm(const float* g, int64_t n, float max_norm, float* coef, double* norm, void* ws,
                         size_t ws_bytes, hipStream_t stream) {
  if (n < 0) return QLORA_ERR_SHAPE;
  if (!(max_norm > 0.0f) || isnan(max_norm)) return QLORA_ERR_ARG;
  if ((n > 0 && !g) || (!coef && !norm)) return QLORA_ERR_ARG;
  if (!ws || ws_bytes < QLORA_CLIP_WORKSPACE_BYTES) return QLORA_ERR_WORKSPACE;
  if (!aligned16(g) || !aligned16(ws) || (reinterpret_cast<uintptr_t>(coef) & 3u) ||
      (reinterpret_cast<uintptr_t>(norm) & 7u))
    return QLORA_ERR_ALIGN;
  const float* gd = n > 0 ? static_cast<const float*>(device_view(g)) : g;
  float* cd = coef ? static_cast<float*>(device_view(coef)) : nullptr;
  double* nd = norm ? static_cast<double*>(device_view(norm)) : nullptr;
  double* wd = static_cast<double*>(device_view(ws));
  if ((n > 0 && !gd) || (coef && !cd) || (norm && !nd) || !wd) return QLORA_ERR_ARG;
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e = qlora::launch_clip_norm(gd, n, (double)max_norm, cd, nd, wd, stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

int qlora_adam_step(float* theta, const float* g, float* m, float* v, int64_t n, const qlora_adam_params* hp,
                    const float* coef, uint16_t* theta_bf16, hipStream_t stream) {
  if (!hp) return QLORA_ERR_ARG;
  if (n < 0) return QLORA_ERR_SHAPE;
  if (!valid_adam(hp)) return QLORA_ERR_ARG;
  if (n == 0) return QLORA_OK;
  if (!theta || !g || !m || !v) return QLORA_ERR_ARG;
  if (!aligned16(theta) || !aligned16(g) || !aligned16(m) || !aligned16(v) || !aligned16(theta_bf16) ||
      (reinterpret_cast<uintptr_t>(coef) & 3u))
    return QLORA_ERR_ALIGN;
  float* td = static_cast<float*>(device_view(theta));
  const float* gd = static_cast<const float*>(device_view(g));
  float* md = static_cast<float*>(device_view(m));
  float* vd = static_cast<float*>(device_view(v));
  const float* cd = coef ? static_cast<const float*>(device_view(coef)) : nullptr;
  uint16_t* bd = theta_bf16 ? static_cast<uint16_t*>(device_view(theta_bf16)) : nullptr;
  if (!td || !gd || !md || !vd || (coef && !cd) || (theta_bf16 && !bd)) return QLORA_ERR_ARG;
  const qlora::AdamHyper h = adam_hyper(hp);
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e = qlora::launch_adam(td, gd, md, vd, n, h, cd, bd, stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

int qlora_adam_state_numel(int n, const int64_t* numel, int64_t* total) {
  if (n < 0 || (n > 0 && !numel) || !total) return QLORA_ERR_ARG;
  int64_t sum = 0;
  for (int k = 0; k < n; ++k) {
    if (numel[k] < 0 || numel[k] > kMaxNumel) return QLORA_ERR_SHAPE;
    sum += qlora::adam_state_span(numel[k]);
    if (sum > kMaxNumel) return QLORA_ERR_SHAPE;
  }
  *total = sum;
  return QLORA_OK;
}

int qlora_clip_grad_norm_batch(int n, const void* const* g, qlora_dtype grad_dtype, const int64_t* numel,
                               float max_norm, float* coef, double* norm, void* ws, size_t ws_bytes,
                               hipStream_t stream) {
  int64_t total = 0;
  const int st = qlora_adam_state_numel(n, numel, &total);
  if (st != QLORA_OK) return st;
  if (grad_dtype != QLORA_F32 && grad_dtype != QLORA_BF16) return QLORA_ERR_ARG;
  if (!(max_norm > 0.0f)) return QLORA_ERR_ARG;
  if ((n > 0 && !g) || (!coef && !norm)) return QLORA_ERR_ARG;
  if (!ws || ws_bytes < QLORA_CLIP_WORKSPACE_BYTES) return QLORA_ERR_WORKSPACE;
  for (int k = 0; k < n; ++k) {
    if (numel[k] > 0 && !g[k]) return QLORA_ERR_ARG;
    if (numel[k] > 0 && !aligned16(g[k])) return QLORA_ERR_ALIGN;
  }
  if (!aligned16(ws) || (reinterpret_cast<uintptr_t>(coef) & 3u) || (reinterpret_cast<uintptr_t>(norm) & 7u))
    return QLORA_ERR_ALIGN;
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e = qlora::launch_clip_norm_batch(n, g, grad_dtype == QLORA_BF16, numel, (double)max_norm, coef,
                                                     norm, static_cast<double*>(ws), stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

int qlora_adamw_batch(int n, float* const* theta, const void* const* g, qlora_dtype grad_dtype,
                      uint16_t* const* theta_bf16, const int64_t* numel, const qlora_adam_state* state,
                      const qlora_adam_params* hp, const float* coef, hipStream_t stream) {
  if (!state || !valid_adam(hp)) return QLORA_ERR_ARG;
  if ((state->bits != 8 && state->bits != 32) || (grad_dtype != QLORA_F32 && grad_dtype != QLORA_BF16))
    return QLORA_ERR_ARG;
  int64_t total = 0;
  const int st = qlora_adam_state_numel(n, numel, &total);
  if (st != QLORA_OK) return st;
  if (total == 0) return QLORA_OK;
  if (!theta || !g || !state->m || !state->v) return QLORA_ERR_ARG;
  if (state->bits == 8 && (!state->m_scale || !state->v_scale)) return QLORA_ERR_ARG;
  for (int k = 0; k < n; ++k) {
    if (numel[k] == 0) continue;
    if (!theta[k] || !g[k] || (theta_bf16 && !theta_bf16[k])) return QLORA_ERR_ARG;
    if (!aligned16(theta[k]) || !aligned16(g[k]) || (theta_bf16 && !aligned16(theta_bf16[k]))) return QLORA_ERR_ALIGN;
  }
  if (!aligned16(state->m) || !aligned16(state->v) || (reinterpret_cast<uintptr_t>(state->m_scale) & 3u) ||
      (reinterpret_cast<uintptr_t>(state->v_scale) & 3u) || (reinterpret_cast<uintptr_t>(coef) & 3u))
    return QLORA_ERR_ALIGN;
  // the state may sit in pinned host memory, as for qlora_adam_step
  qlora::AdamBatch b;
  b.n = n;
  b.theta = theta;
  b.g = g;
  b.g16 = grad_dtype == QLORA_BF16;
  b.theta16 = theta_bf16;
  b.numel = numel;
  b.bits8 = state->bits == 8;
  b.m = device_view(state->m);
  b.v = device_view(state->v);
  b.m_scale = b.bits8 ? static_cast<float*>(device_view(state->m_scale)) : nullptr;
  b.v_scale = b.bits8 ? static_cast<float*>(device_view(state->v_scale)) : nullptr;
  if (!b.m || !b.v || (b.bits8 && (!b.m_scale || !b.v_scale))) return QLORA_ERR_ARG;
  const qlora::AdamHyper h = adam_hyper(hp);
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e = qlora::launch_adamw_batch(b, h, coef, stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

// Arguments shared by the linears with an adapter per row (every pointer but
// the workspace that must be there and aligned; counts last).
static int check_multi(const qlora_nf4* W, const void* X, int64_t M, const int32_t* row_adapter, int n_adapters,
                       const void* L1, const void* L2, int r, const float* scale) {
  const int st = check_linear(W, M, r, 1.0f);
  if (st != QLORA_OK) return st;
  if (n_adapters < 1 || n_adapters > QLORA_MULTI_MAX_ADAPTERS || !L1 || !L2 || !scale) return QLORA_ERR_ARG;
  if (M > QLORA_MULTI_MAX_ROWS) return QLORA_ERR_SHAPE;
  if (M > 0 && (!X || !row_adapter)) return QLORA_ERR_ARG;
  if (!aligned16(X) || !aligned16(L1) || !aligned16(L2) || (reinterpret_cast<uintptr_t>(row_adapter) & 3u) ||
      (reinterpret_cast<uintptr_t>(scale) & 3u))
    return QLORA_ERR_ALIGN;
  return QLORA_OK;
}

int qlora_linear_multi_workspace(int64_t M, int64_t K, int64_t N, int r, int n_adapters, int backward,
                                 size_t* bytes) {
  if (!bytes || n_adapters < 1 || n_adapters > QLORA_MULTI_MAX_ADAPTERS) return QLORA_ERR_ARG;
  const int st = qlora_linear_workspace(M < 0 ? -1 : 0, K, N, r, bytes);   // the rules of the single linear
  if (st != QLORA_OK) return st;
  if (M > QLORA_MULTI_MAX_ROWS) return QLORA_ERR_SHAPE;
  *bytes = qlora::multi_workspace_layout(M, K, N, r, n_adapters, backward != 0).total;
  return QLORA_OK;
}

int qlora_linear_multi_fwd(const qlora_nf4* W, const uint16_t* X, int64_t M, const int32_t* row_adapter,
                           int n_adapters, const uint16_t* L1, const uint16_t* L2, int r, const float* scale,
                           uint16_t* Y, uint16_t* T_out, void* ws, size_t ws_bytes, hipStream_t stream) {
  const int st = check_multi(W, X, M, row_adapter, n_adapters, L1, L2, r, scale);
  if (st != QLORA_OK) return st;
  if (M == 0) return QLORA_OK;
  if (!Y) return QLORA_ERR_ARG;
  if (!ws) return QLORA_ERR_WORKSPACE;
  if (!aligned16(Y) || !aligned16(T_out) || !aligned16(ws)) return QLORA_ERR_ALIGN;
  if (!qlora::multi_forward_supported(M, W->cols, W->rows, r, n_adapters)) return QLORA_ERR_SHAPE;
  if (ws_bytes < qlora::multi_workspace_layout(M, W->cols, W->rows, r, n_adapters, false).total)
    return QLORA_ERR_WORKSPACE;
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e = qlora::multi_forward(view_of(W), tables(W->qtype).tab, X, M, row_adapter, n_adapters, L1, L2,
                                            r, scale, Y, T_out, ws, stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

int qlora_linear_multi_bwd(const qlora_nf4* W, const uint16_t* X, const uint16_t* dY, int64_t M,
                           const int32_t* row_adapter, int n_adapters, const uint16_t* L1, const uint16_t* L2, int r,
                           const float* scale, const uint16_t* T, uint16_t* dX, void* dL1, void* dL2,
                           qlora_dtype grad_dtype, void* ws, size_t ws_bytes, hipStream_t stream) {
  const int st = check_multi(W, X, M, row_adapter, n_adapters, L1, L2, r, scale);
  if (st != QLORA_OK) return st;
  if (grad_dtype != QLORA_F32 && grad_dtype != QLORA_BF16) return QLORA_ERR_ARG;
  if (!dL1 || !dL2 || (M > 0 && !dY)) return QLORA_ERR_ARG;
  if (!ws) return QLORA_ERR_WORKSPACE;
  if (!aligned16(dY) || !aligned16(T) || !aligned16(dX) || !aligned16(dL1) || !aligned16(dL2) || !aligned16(ws))
    return QLORA_ERR_ALIGN;
  if (!qlora::multi_dense_supported(W->cols, W->rows, r)) return QLORA_ERR_SHAPE;
  if (dX && !qlora::multi_lay_supported(M, W->cols, r, n_adapters, false)) return QLORA_ERR_SHAPE;
  if (ws_bytes < qlora::multi_workspace_layout(M, W->cols, W->rows, r, n_adapters, true).total)
    return QLORA_ERR_WORKSPACE;
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e =
      qlora::multi_backward(view_of(W), tables(W->qtype).tab, X, dY, M, row_adapter, n_adapters, L1, L2, r, scale, T,
                            dX, dL1, dL2, grad_dtype == QLORA_BF16, ws, stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

// Shapes of a preference loss: S T rows of V logits; rows is S T.
static int check_preference(int64_t pairs, int64_t T, int64_t V, int64_t* rows) {
  if (pairs < 0 || T < 0 || V < 1 || pairs > ((int64_t)1 << 20) || T > ((int64_t)1 << 30) || V > ((int64_t)1 << 30))
    return QLORA_ERR_SHAPE;
  *rows = 2 * pairs * T;
  return *rows > 0x7FFFFFFF ? QLORA_ERR_SHAPE : QLORA_OK;
}

int qlora_preference_workspace(int64_t pairs, int64_t T, int64_t V, size_t* bytes) {
  if (!bytes) return QLORA_ERR_ARG;
  int64_t rows = 0;
  const int st = check_preference(pairs, T, V, &rows);
  if (st != QLORA_OK) return st;
  *bytes = qlora::pref_workspace_layout(pairs, T).total;
  return QLORA_OK;
}

int qlora_preference_loss(const void* logits, qlora_dtype dtype, int64_t pairs, int64_t T, int64_t V, int64_t ld,
                          const int64_t* labels, const float* ref_logps, float beta, float label_smoothing,
                          float grad_scale, float* loss, float* rewards, float* logps, void* dlogits, int64_t ldd,
                          void* ws, size_t ws_bytes, hipStream_t stream) {
  if (dtype != QLORA_F32 && dtype != QLORA_BF16) return QLORA_ERR_ARG;
  if (!isfinite(beta) || !isfinite(grad_scale) || !(label_smoothing >= 0.0f && label_smoothing <= 1.0f))
    return QLORA_ERR_ARG;
  int64_t rows = 0;
  size_t need = 0;
  int st = check_preference(pairs, T, V, &rows);
  if (st != QLORA_OK) return st;
  if (ld < V || (dlogits && ldd < V)) return QLORA_ERR_SHAPE;
  if (dlogits == logits && dlogits && ldd != ld) return QLORA_ERR_SHAPE;   // in place: the same rows
  if (!loss || (pairs > 0 && !rewards) || (rows > 0 && (!logits || !labels || !ref_logps || !logps)))
    return QLORA_ERR_ARG;
  st = qlora_preference_workspace(pairs, T, V, &need);
  if (st != QLORA_OK) return st;
  if (!ws || ws_bytes < need) return QLORA_ERR_WORKSPACE;
  const uintptr_t elem = dtype == QLORA_F32 ? 3u : 1u;
  const auto off = [](const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; };
  if (off(logits, elem) || off(dlogits, elem) || off(labels, 7u) || off(ref_logps, 3u) || off(loss, 3u) ||
      off(rewards, 3u) || off(logps, 3u) || !aligned16(ws))
    return QLORA_ERR_ALIGN;
  qlora::PrefCall c;
  c.logits = logits;
  c.bf16 = dtype == QLORA_BF16;
  c.labels = labels;
  c.ref = ref_logps;
  c.S = (int)(2 * pairs);
  c.T = (int)T;
  c.V = (int)V;
  c.ld = ld;
  c.ldd = ldd;
  c.beta = beta;
  c.eps = label_smoothing;
  c.gscale = grad_scale;
  c.loss = loss;
  c.rewards = rewards;
  c.logps = logps;
  c.dlogits = dlogits;
  c.ws = ws;
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e = qlora::launch_preference(c, stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

// ---- the rest of a training step (qlora_layers.h) ----------------------------------------------

static bool off_by(const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

// Optional int8 values: absent, or both buffers there (QLORA_OK), aligned.
static int check_int8(const qlora_int8_values* v, bool rows) {
  if (!v || !rows) return QLORA_OK;
  if (!v->codes || !v->absmax) return QLORA_ERR_ARG;
  return aligned16(v->codes) && !off_by(v->absmax, 3u) ? QLORA_OK : QLORA_ERR_ALIGN;
}

static qlora::Int8Values int8_of(const qlora_int8_values* v) {
  return v ? qlora::Int8Values{v->codes, v->absmax} : qlora::Int8Values{nullptr, nullptr};
}

static int check_layer_shape(int64_t M, int64_t K, int64_t F, int r) {
  if (r < 8 || r > QLORA_MAX_RANK || (r % 8) != 0) return QLORA_ERR_ARG;
  if (M < 0 || K <= 0 || F <= 0 || (K % QLORA_BLOCK) != 0 || (F % 8) != 0) return QLORA_ERR_SHAPE;
  if (M > QLORA_LAYER_MAX_ROWS || K >= QLORA_GATED_MAX_COLS || F >= QLORA_GATED_MAX_COLS) return QLORA_ERR_SHAPE;
  return QLORA_OK;
}

int qlora_gated_workspace(int64_t M, int64_t K, int64_t F, int r, int backward, size_t* bytes) {
  if (!bytes) return QLORA_ERR_ARG;
  const int st = check_layer_shape(M, K, F, r);
  if (st != QLORA_OK) return st;
  *bytes = qlora::gated_workspace_layout(M, K, F, r, backward != 0).total;
  return QLORA_OK;
}

// The arguments that both passes share.
static int check_gated(const qlora_nf4* gate, const qlora_nf4* up, int64_t M, const void* L1, const void* L2, int r,
                       float scale, qlora_act act, const void* T, const qlora_int8_values* gate8,
                       const qlora_int8_values* up8) {
  if (!valid_nf4(gate) || !valid_nf4(up) || !isfinite(scale)) return QLORA_ERR_ARG;
  if (act != QLORA_ACT_SILU && act != QLORA_ACT_GELU_TANH) return QLORA_ERR_ARG;
  if (gate->rows != up->rows || gate->cols != up->cols) return QLORA_ERR_SHAPE;
  int st = check_layer_shape(M, gate->cols, gate->rows, r);
  if (st != QLORA_OK) return st;
  if (!L1 || !L2 || (gate8 == nullptr) != (up8 == nullptr)) return QLORA_ERR_ARG;
  if (gate8 && gate->rows % QLORA_BLOCK != 0) return QLORA_ERR_SHAPE;
  st = check_int8(gate8, M > 0);
  if (st == QLORA_OK) st = check_int8(up8, M > 0);
  if (st != QLORA_OK) return st;
  if (!aligned16(gate->codes) || !aligned16(up->codes) || !aligned16(L1) || !aligned16(L2) || !aligned16(T))
    return QLORA_ERR_ALIGN;
  return QLORA_OK;
}

static qlora::GatedBase gated_base(const qlora_nf4* gate, const qlora_nf4* up) {
  return qlora::GatedBase{view_of(gate), view_of(up), tables(gate->qtype).tab, tables(up->qtype).tab};
}

int qlora_gated_fwd(const qlora_nf4* gate, const qlora_nf4* up, const uint16_t* X, int64_t M, const uint16_t* L1,
                    const uint16_t* L2, int r, float scale, qlora_act act, uint16_t* A, uint16_t* T_out,
                    const qlora_int8_values* gate8, const qlora_int8_values* up8, void* ws, size_t ws_bytes,
                    hipStream_t stream) {
  const int st = check_gated(gate, up, M, L1, L2, r, scale, act, T_out, gate8, up8);
  if (st != QLORA_OK) return st;
  if (M == 0) return QLORA_OK;
  if (!X || !A) return QLORA_ERR_ARG;
  if (!ws) return QLORA_ERR_WORKSPACE;
  if (!aligned16(X) || !aligned16(A) || !aligned16(ws)) return QLORA_ERR_ALIGN;
  if (ws_bytes < qlora::gated_workspace_layout(M, gate->cols, gate->rows, r, false).total) return QLORA_ERR_WORKSPACE;
  const qlora::Int8Values g8 = int8_of(gate8), u8 = int8_of(up8);
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e = qlora::gated_forward(gated_base(gate, up), X, M, L1, L2, r, scale, (int)act, A, T_out,
                                            gate8 ? &g8 : nullptr, up8 ? &u8 : nullptr, ws, stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

int qlora_gated_bwd(const qlora_nf4* gate, const qlora_nf4* up, const uint16_t* X, const qlora_int8_values* X8,
                    const uint16_t* dA, int64_t M, const uint16_t* L1, const uint16_t* L2, int r, float scale,
                    qlora_act act, const uint16_t* T, const qlora_int8_values* gate8, const qlora_int8_values* up8,
                    uint16_t* dX, void* dL1, void* dL2, qlora_dtype grad_dtype, void* ws, size_t ws_bytes,
                    hipStream_t stream) {
  int st = check_gated(gate, up, M, L1, L2, r, scale, act, T, gate8, up8);
  if (st != QLORA_OK) return st;
  if (grad_dtype != QLORA_F32 && grad_dtype != QLORA_BF16) return QLORA_ERR_ARG;
  if (!dL1 || !dL2 || (M > 0 && (!dA || (X == nullptr) == (X8 == nullptr)))) return QLORA_ERR_ARG;
  st = check_int8(X8, M > 0);
  if (st != QLORA_OK) return st;
  if (!ws) return QLORA_ERR_WORKSPACE;
  if (!aligned16(X) || !aligned16(dA) || !aligned16(dX) || !aligned16(dL1) || !aligned16(dL2) || !aligned16(ws))
    return QLORA_ERR_ALIGN;
  if (ws_bytes < qlora::gated_workspace_layout(M, gate->cols, gate->rows, r, true).total) return QLORA_ERR_WORKSPACE;
  const qlora::Int8Values g8 = int8_of(gate8), u8 = int8_of(up8), x8 = int8_of(X8);
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e = qlora::gated_backward(gated_base(gate, up), X, X8 ? &x8 : nullptr, dA, M, L1, L2, r, scale,
                                             (int)act, T, gate8 ? &g8 : nullptr, up8 ? &u8 : nullptr, dX, dL1, dL2,
                                             grad_dtype == QLORA_BF16, ws, stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

int qlora_linear_bwd_int8_workspace(int64_t M, int64_t K, int64_t N, int r, size_t* bytes) {
  if (!bytes) return QLORA_ERR_ARG;
  const int st = check_layer_shape(M, K, N, r);
  if (st != QLORA_OK) return st;
  *bytes = qlora::linear_int8_workspace_layout(M, K, N, r).total;
  return QLORA_OK;
}

int qlora_linear_bwd_int8(const qlora_nf4* W, const qlora_int8_values* X8, const uint16_t* dY, int64_t M,
                          const uint16_t* L1, const uint16_t* L2, int r, float scale, const uint16_t* T, uint16_t* dX,
                          void* dL1, void* dL2, qlora_dtype grad_dtype, void* ws, size_t ws_bytes,
                          hipStream_t stream) {
  int st = check_linear(W, M, r, scale);
  if (st == QLORA_OK) st = check_layer_shape(M, W->cols, W->rows, r);
  if (st != QLORA_OK) return st;
  if (grad_dtype != QLORA_F32 && grad_dtype != QLORA_BF16) return QLORA_ERR_ARG;
  if (!L1 || !L2 || !dL1 || !dL2 || (M > 0 && (!X8 || !dY))) return QLORA_ERR_ARG;
  st = check_int8(X8, M > 0);
  if (st != QLORA_OK) return st;
  if (!ws) return QLORA_ERR_WORKSPACE;
  if (!aligned16(dY) || !aligned16(L1) || !aligned16(L2) || !aligned16(T) || !aligned16(dX) || !aligned16(dL1) ||
      !aligned16(dL2) || !aligned16(ws))
    return QLORA_ERR_ALIGN;
  if (ws_bytes < qlora::linear_int8_workspace_layout(M, W->cols, W->rows, r).total) return QLORA_ERR_WORKSPACE;
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e = qlora::linear_backward_int8(view_of(W), tables(W->qtype).tab, int8_of(X8), dY, M, L1, L2, r, scale, T,
                                                   dX, dL1, dL2, grad_dtype == QLORA_BF16, ws, stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

static int check_norm(int64_t M, int64_t K, qlora_dtype a, qlora_dtype b, qlora_dtype c) {
  for (qlora_dtype t : {a, b, c})
    if (t != QLORA_F32 && t != QLORA_BF16) return QLORA_ERR_ARG;
  if (M < 0 || M > QLORA_LAYER_MAX_ROWS || K < 8 || K > QLORA_NORM_MAX_COLS || (K % 8) != 0) return QLORA_ERR_SHAPE;
  return QLORA_OK;
}

int qlora_norm_workspace(int64_t M, int64_t K, size_t* bytes) {
  if (!bytes) return QLORA_ERR_ARG;
  const int st = check_norm(M, K, QLORA_F32, QLORA_F32, QLORA_F32);
  if (st != QLORA_OK) return st;
  *bytes = qlora::align_up((size_t)qlora::norm_slices(M) * (size_t)K * 4 + 1, 256);
  return QLORA_OK;
}

int qlora_norm_fwd(const void* x, qlora_dtype x_dtype, const void* residual, qlora_dtype stream_dtype,
                   const void* weight, qlora_dtype weight_dtype, int64_t M, int64_t K, float eps, uint16_t* y,
                   const qlora_int8_values* y8, void* h, float* rstd, hipStream_t stream) {
  int st = check_norm(M, K, x_dtype, residual ? stream_dtype : x_dtype, weight ? weight_dtype : x_dtype);
  if (st != QLORA_OK) return st;
  if (!isfinite(eps) || eps < 0.0f) return QLORA_ERR_ARG;
  if (y8 && K % QLORA_BLOCK != 0) return QLORA_ERR_SHAPE;
  if (M == 0) return QLORA_OK;
  if (!x || (residual == nullptr) != (h == nullptr)) return QLORA_ERR_ARG;
  st = check_int8(y8, true);
  if (st != QLORA_OK) return st;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(y) || !aligned16(h) || off_by(rstd, 3u))
    return QLORA_ERR_ALIGN;
  qlora::NormFwd c{};
  c.x = x;
  c.res = residual;
  c.x_bf16 = x_dtype == QLORA_BF16;
  c.res_bf16 = stream_dtype == QLORA_BF16;
  c.w = weight;
  c.w_bf16 = weight_dtype == QLORA_BF16;
  c.M = M;
  c.K = K;
  c.eps = eps;
  c.y = y;
  c.codes = y8 ? y8->codes : nullptr;
  c.absmax = y8 ? y8->absmax : nullptr;
  c.h = h;
  c.rstd = rstd;
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e = qlora::launch_norm_fwd(c, stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

int qlora_norm_bwd(const uint16_t* dy, const void* h, qlora_dtype stream_dtype, const float* rstd, const void* weight,
                   qlora_dtype weight_dtype, const void* dres, int64_t M, int64_t K, void* dh, uint16_t* dx16,
                   float* dweight, void* ws, size_t ws_bytes, hipStream_t stream) {
  const int st = check_norm(M, K, stream_dtype, stream_dtype, weight ? weight_dtype : stream_dtype);
  if (st != QLORA_OK) return st;
  if (M > 0 && (!dy || !h || !rstd || !dh)) return QLORA_ERR_ARG;
  if (!aligned16(dy) || !aligned16(h) || off_by(rstd, 3u) || !aligned16(weight) || !aligned16(dres) || !aligned16(dh) ||
      !aligned16(dx16) || off_by(dweight, 3u) || !aligned16(ws))
    return QLORA_ERR_ALIGN;
  if (dweight) {
    size_t need = 0;
    qlora_norm_workspace(M, K, &need);
    if (!ws || ws_bytes < need) return QLORA_ERR_WORKSPACE;
  }
  qlora::NormBwd c{};
  c.dy = dy;
  c.h = h;
  c.h_bf16 = stream_dtype == QLORA_BF16;
  c.rstd = rstd;
  c.w = weight;
  c.w_bf16 = weight_dtype == QLORA_BF16;
  c.dres = dres;
  c.M = M;
  c.K = K;
  c.dh = dh;
  c.dx16 = dx16;
  c.dw = dweight;
  c.part = static_cast<float*>(ws);
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e = qlora::launch_norm_bwd(c, stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

static int check_head(int64_t M, int64_t K, int64_t V, qlora_dtype grad_dtype) {
  if (grad_dtype != QLORA_F32 && grad_dtype != QLORA_BF16) return QLORA_ERR_ARG;
  if (M < 0 || M > QLORA_LAYER_MAX_ROWS || K <= 0 || (K % 64) != 0 || K >= ((int64_t)1 << 23) || V < 1 ||
      V > QLORA_HEAD_MAX_VOCAB)
    return QLORA_ERR_SHAPE;
  return QLORA_OK;
}

int qlora_head_workspace(int64_t M, int64_t K, int64_t V, int dH, int dW, qlora_dtype grad_dtype, size_t* bytes) {
  if (!bytes) return QLORA_ERR_ARG;
  const int st = check_head(M, K, V, grad_dtype);
  if (st != QLORA_OK) return st;
  *bytes = qlora::head_workspace_layout(M, K, V, dH != 0, dW != 0, grad_dtype == QLORA_BF16).total;
  return QLORA_OK;
}

int qlora_head_loss(const uint16_t* H, const uint16_t* W, const int64_t* labels, const float* weights, int64_t M,
                    int64_t K, int64_t V, float divisor, float grad_scale, float* loss, float* nll, uint16_t* dH,
                    void* dW, qlora_dtype grad_dtype, void* ws, size_t ws_bytes, hipStream_t stream) {
  const int st = check_head(M, K, V, grad_dtype);
  if (st != QLORA_OK) return st;
  if (!isfinite(divisor) || divisor < 0.0f || !isfinite(grad_scale)) return QLORA_ERR_ARG;
  if (!W || !loss || (M > 0 && (!H || !labels || !nll))) return QLORA_ERR_ARG;
  if (!aligned16(H) || !aligned16(W) || off_by(labels, 7u) || off_by(weights, 3u) || off_by(loss, 3u) || off_by(nll, 3u) ||
      !aligned16(dH) || !aligned16(dW) || !aligned16(ws))
    return QLORA_ERR_ALIGN;
  if (!ws || ws_bytes < qlora::head_workspace_layout(M, K, V, dH != nullptr, dW != nullptr, grad_dtype == QLORA_BF16).total)
    return QLORA_ERR_WORKSPACE;
  qlora::HeadCall c{};
  c.H = H;
  c.W = W;
  c.labels = labels;
  c.weights = weights;
  c.M = M;
  c.K = K;
  c.V = V;
  c.divisor = divisor;
  c.grad_scale = grad_scale;
  c.loss = loss;
  c.nll = nll;
  c.dH = dH;
  c.dW = dW;
  c.dw_bf16 = grad_dtype == QLORA_BF16;
  c.ws = ws;
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e = qlora::launch_head_loss(c, stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

int qlora_lora_dropout(const uint16_t* X, int64_t numel, float p, uint64_t seed, uint16_t* Xd, hipStream_t stream) {
  if (!valid_dropout(p)) return QLORA_ERR_ARG;
  if (numel < 0 || (numel % 8) != 0 || numel > ((int64_t)1 << 40)) return QLORA_ERR_SHAPE;
  if (numel == 0) return QLORA_OK;
  if (!X || !Xd) return QLORA_ERR_ARG;
  if (!aligned16(X) || !aligned16(Xd)) return QLORA_ERR_ALIGN;
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e = qlora::launch_dropout_input(X, numel, qlora::dropout_params(p, seed), Xd, stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

int qlora_check_conversions(uint32_t first, int64_t count, uint16_t* bf16_out, uint8_t* e4m3_out,
                            float* e4m3_table, hipStream_t stream) {
  if (count < 0 || count > ((int64_t)1 << 32)) return QLORA_ERR_SHAPE;
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e = qlora::launch_convcheck(first, count, bf16_out, e4m3_out, e4m3_table, stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

int qlora_probe_mfma(int workgroups, int iters, float* sink, uint64_t* clocks, hipStream_t stream) {
  if (!sink || !clocks || workgroups < 1 || workgroups > (1 << 20) || iters < 1 || iters > (1 << 20))
    return QLORA_ERR_ARG;
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e = qlora::launch_mfma_probe(workgroups, iters, sink,
                                                reinterpret_cast<unsigned long long*>(clocks), stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

int qlora_probe_read(const void* src, size_t bytes, uint32_t never, uint32_t* sink, hipStream_t stream) {
  static_assert(QLORA_PROBE_READ_GRANULE == 65536, "granule");
  if (bytes == 0 || bytes % qlora::read_probe_granule() != 0 || bytes >= ((size_t)1 << 40)) return QLORA_ERR_SHAPE;
  if (!src || !sink) return QLORA_ERR_ARG;
  if (!aligned16(src)) return QLORA_ERR_ALIGN;
  (void)hipGetLastError();  // drop an error left by an earlier, unrelated runtime call
  const hipError_t e = qlora::launch_read_probe(src, bytes, never, sink, stream);
  return e == hipSuccess ? QLORA_OK : hip_fail(e);
}

int qlora_set_timing(int kernel, hipEvent_t* start, hipEvent_t* stop, int n, int* count) {
  if (kernel < 0 || kernel >= QLORA_TIMING_CLASSES || n < 0) return QLORA_ERR_ARG;
  qlora::TimingSlot& t = qlora::timing_slots()[kernel];
  if (n == 0 || !start || !stop || !count) {
    t = qlora::TimingSlot();
    return QLORA_OK;
  }
  t.start = start;
  t.stop = stop;
  t.n = n;
  t.count = count;
  return QLORA_OK;
}

}  // extern "C"

namespace qlora {
TimingSlot* timing_slots() {
  static thread_local TimingSlot slots[kTimeClasses];
  return slots;
}
}  // namespace qlora
