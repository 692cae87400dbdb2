/*
 * qlora_adapters.h -- many adapters on one quantised base: the C ABI of the
 * entry points beside qlora_nf4.h (same library, same conventions, status
 * codes, types and workspace rules).
 *
 *   - qlora_linear_multi_fwd / _bwd: the QLoRA linear with an adapter per row;
 *   - qlora_preference_loss: a preference loss over pairs of sequences, with
 *     the gradient of the logits;
 *   - qlora_clip_grad_norm_batch / qlora_adamw_batch: the optimiser step over
 *     all adapter tensors at once, with fp32 or 8-bit state.
 */
#ifndef QLORA_ADAPTERS_H
#define QLORA_ADAPTERS_H

#include "qlora_nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The QLoRA linear with an adapter per row: several adapters of one rank, and
 * rows without any, beside one frozen weight, in one call. With a =
 * row_adapter[m],
 *   Y[m]  = X[m] dequant(Wt)^T + scale[a] (X[m] L1[a]) L2[a]     (the base alone for a outside [0, n_adapters))
 *   dX[m] = dY[m] dequant(Wt) + scale[a] (dY[m] L2[a]^T) L1[a]^T
 *   dL1[a] = scale[a] sum over the rows m of a of X[m]^T (dY[m] L2[a]^T)
 *   dL2[a] = scale[a] sum over the rows m of a of (X[m] L1[a])^T dY[m]
 * computed as qlora_linear_fwd / _bwd compute them for one adapter (bf16
 * operands, fp32 accumulation; s T and s U are rounded to bf16 before their
 * second product, outputs once). Rows may come in any order. An adapter
 * without rows gets zero gradients. Sums run in a fixed order. Infinities and
 * NaN of one row or one adapter reach no other row and no other adapter's
 * gradients. (Within a row whose s T or s U holds an infinity, its product with
 * an infinity of the adapter's second factor may come out as NaN.) Up to 16
 * rows may take paths that hold the code values in fp16, so that some weights
 * are the neighbouring bf16 of the dequantised ones (2.7 % for NF4). There is no
 * LoRA dropout here.
 *   W            host struct of the quantised weight [N][K].
 *   X            device bf16 [M][K];  dY device bf16 [M][N].
 *   row_adapter  device int32 [M].
 *   n_adapters   A, 1 .. QLORA_MULTI_MAX_ADAPTERS; adapters of a smaller rank
 *                are padded with zero columns of L1 and rows of L2.
 *   L1, L2       device bf16 [A][K][r], [A][r][N];  scale device fp32 [A].
 *   T_out, T     optional device bf16 [M][r] = bf16(X[m] L1[a]), zero for rows
 *                without an adapter: written by the forward pass, read by the
 *                backward pass (which computes it when T is NULL).
 *   dX           device bf16 [M][K], or NULL to skip it.
 *   dL1, dL2     device, grad_dtype, shaped like L1, L2.
 *   ws           qlora_linear_multi_workspace(M, K, N, r, A, backward) bytes,
 *                which never shrink as M grows: one of the largest batch's
 *                size serves smaller batches.
 * Shape rules as for qlora_linear_fwd (K a multiple of 64, N and r of 8, r in
 * [8, 256]), M <= QLORA_MULTI_MAX_ROWS; M > 128 and the backward pass need a
 * dequantised weight below 2 GB, and the factor that the GEMM lays out for the
 * adapters with rows (L2 in the forward pass, L1 for dX) below about 64 GB, its
 * rank rounded up to 64: QLORA_ERR_SHAPE otherwise. M <= 128 streams the 4-bit
 * weight once, and a single token (or, for r <= 64, a few) takes the GEMV.
 */
#define QLORA_MULTI_MAX_ROWS (1 << 22)
#define QLORA_MULTI_MAX_ADAPTERS 4096
int qlora_linear_multi_workspace(int64_t M, int64_t K, int64_t N, int r, int n_adapters, int backward,
                                 size_t *bytes);
int qlora_linear_multi_fwd(const qlora_nf4 *W, const uint16_t *X, int64_t M, const int32_t *row_adapter,
                           int n_adapters, const uint16_t *L1, const uint16_t *L2, int r, const float *scale,
                           uint16_t *Y, uint16_t *T_out, void *ws, size_t ws_bytes, hipStream_t stream);
int qlora_linear_multi_bwd(const qlora_nf4 *W, const uint16_t *X, const uint16_t *dY, int64_t M,
                           const int32_t *row_adapter, int n_adapters, const uint16_t *L1, const uint16_t *L2, int r,
                           const float *scale, const uint16_t *T, uint16_t *dX, void *dL1, void *dL2,
                           qlora_dtype grad_dtype, void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * qlora_preference_loss: a loss over pairs of sequences from the paired log
 * ratios of a policy and a reference, and the gradient of the policy's logits
 * (Rafailov et al., "Direct Preference Optimization", NeurIPS 2023, eq. 7).
 * Sequences s = 0 .. pairs - 1 are the preferred ones, s + pairs the other one
 * of the same pair; S = 2 pairs.
 *   lp[s][t]  = logits[s][t][y] - log sum_v exp(logits[s][t][v]),  y = labels[s][t]
 *   reward[s] = beta sum_t (lp[s][t] - ref_logps[s][t]) over the counted t
 *   h_p       = reward[p] - reward[pairs + p]
 *   loss      = 1 / pairs sum_p (1 - e) softplus(-h_p) + e softplus(h_p)   (0 without pairs)
 *   dlogits   = grad_scale d loss / d logits
 * A position counts when its label lies in [0, V); the others' logits and
 * references are not used, their lp is 0 and their gradient rows are zero. A
 * sequence may have no counted position. -inf logits take no probability.
 *   logits     device, dtype, rows [s T + t] of V values, ld >= V elements
 *              apart; any element alignment.
 *   labels     device int64 [S T]: the token that row (s, t) predicts.
 *   ref_logps  device fp32 [S T]: the reference's lp.
 *   label_smoothing  e in [0, 1].  grad_scale: the upstream gradient.
 *   loss [1], rewards [S], logps [S T]: device fp32.
 *   dlogits    device, dtype, rows ldd >= V elements apart, written once; NULL
 *              for the loss alone. It may be logits itself (then ldd == ld), and
 *              otherwise does not overlap them.
 *   ws         qlora_preference_workspace bytes.
 * exp and the sum of a row are fp32 around the row's running maximum, rewards
 * and loss float64 sums in a fixed order, the gradient is rounded once to dtype.
 * Limits: pairs <= 2^20, T and V <= 2^30, S T <= 2^31 - 1.
 */
int qlora_preference_workspace(int64_t pairs, int64_t T, int64_t V, size_t *bytes);
int qlora_preference_loss(const void *logits, qlora_dtype dtype, int64_t pairs, int64_t T, int64_t V, int64_t ld,
                          const int64_t *labels, const float *ref_logps, float beta, float label_smoothing,
                          float grad_scale, float *loss, float *rewards, float *logps, void *dlogits, int64_t ldd,
                          void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * The optimiser step over many tensors at once: the adapters as they were
 * allocated, one (dL1, dL2) pair per linear, with no copy into a flat vector.
 * theta[k], g[k], theta_bf16[k] are host arrays of n device pointers, numel[k]
 * the tensors' sizes (0 .. 2^40; empty tensors are skipped); gradients are all
 * fp32 or all bf16 (grad_dtype). Every tensor is 16-byte aligned, in device
 * memory, and no two overlap. n may be 0. Deterministic; nothing is allocated.
 *
 * qlora_adam_state: the two state vectors of all tensors, one array each:
 * tensor k's values start at element off_k = sum_{j < k} 256 ceil(numel_j / 256),
 * and the arrays hold qlora_adam_state_numel values (the padding behind a
 * tensor is scratch). The arrays may be device or pinned host memory ("paged
 * out", section 方法总览 item 4). Zeros are the state before the first step.
 *   bits 32  m, v: fp32; the scales are not used (may be NULL).
 *   bits 8   m: E4M3 codes (OCP E4M3FN) of the first moment, v: E4M3 codes of
 *            sqrt(second moment); m_scale, v_scale: fp32, one per 256 values.
 *            A value is code * scale. Written per block of 256 as
 *            scale = RN32(top / 448), code = E4M3(RN32(x RN32(448 / top))),
 *            nearest, ties to the even code, top the block's largest magnitude
 *            (below 2^-100: all zeros); a nonzero sqrt(v) gets at least the
 *            smallest code, so that it never leaves eps alone to divide by.
 *
 * qlora_clip_grad_norm_batch: qlora_clip_grad_norm's norm and coef over all
 * tensors' gradients (float64 sums in a fixed order; bf16 gradients are
 * squared exactly). coef, norm, ws as there, in device memory. Gradients with
 * NaN have norm NaN and, as there, coef 1.
 *
 * qlora_adamw_batch: qlora_adam_step's update of every tensor, element by
 * element with the same arithmetic (weight decay decoupled from the moments);
 * with 8 bits, v is the square of the stored root, and theta is stepped with
 * this step's m and v before they are rounded to codes.
 *   theta_bf16  bf16 copies, or NULL for none.
 *   coef        device fp32 [1], or NULL for 1.
 */
typedef struct {
  int32_t bits;
  void *m;
  void *v;
  float *m_scale;
  float *v_scale;
} qlora_adam_state;
int qlora_adam_state_numel(int n, const int64_t *numel, int64_t *total);
int qlora_clip_grad_norm_batch(int n, const void *const *g, qlora_dtype grad_dtype, const int64_t *numel,
                               float max_norm, float *coef, double *norm, void *ws, size_t ws_bytes,
                               hipStream_t stream);
int qlora_adamw_batch(int n, float *const *theta, const void *const *g, qlora_dtype grad_dtype,
                      uint16_t *const *theta_bf16, const int64_t *numel, const qlora_adam_state *state,
                      const qlora_adam_params *hp, const float *coef, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_ADAPTERS_H */
