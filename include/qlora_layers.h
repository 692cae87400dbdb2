/*
 * qlora_layers.h -- the rest of a training step beside the quantised linears:
 * the C ABI of the entry points beside qlora_nf4.h (same library, same
 * conventions, status codes, types and workspace rules).
 *
 *   - qlora_gated_fwd / _bwd: the gated feed-forward block's first half over two
 *     quantised bases with adapters, act(gate) * up;
 *   - qlora_linear_bwd_int8: the linear's backward pass from an input that was
 *     kept in 8 bits;
 *   - qlora_norm_fwd / _bwd: the root-mean-square norm with the residual's
 *     addition, its output in bf16 and in 8 bits;
 *   - qlora_head_loss: softmax cross entropy over the vocabulary from hidden
 *     states and the head's weight, without logits, with its gradients.
 *
 * Activations in 8 bits ("int8 values") are those of qlora_int8_quantize with
 * blocks of 64: codes [numel] and one fp32 absmax per 64 consecutive values, of a
 * matrix whose rows are a multiple of 64 long. A value is code * RN32(absmax / 127).
 * Where these entry points write them, a block that holds an infinity or NaN
 * has that as its absmax and codes 0: its 64 values are NaN.
 * M (rows) is at most QLORA_LAYER_MAX_ROWS, and may be 0. A workspace for M rows serves fewer rows too.
 */
#ifndef QLORA_LAYERS_H
#define QLORA_LAYERS_H

#include "qlora_nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define QLORA_LAYER_MAX_ROWS (1 << 21)
#define QLORA_GATED_MAX_COLS (1 << 22)
#define QLORA_NORM_MAX_COLS 16384
#define QLORA_HEAD_MAX_VOCAB (1 << 22)

typedef struct {
  int8_t *codes;
  float *absmax;
} qlora_int8_values;

typedef enum { QLORA_ACT_SILU = 0, QLORA_ACT_GELU_TANH = 1 } qlora_act;

/*
 * The gated block: with G = X Wg^T + scale (X L1[0]) L2[0] and U = X Wu^T + scale (X L1[1]) L2[1]
 * (Wg, Wu the dequantised weights),
 *   A  = act(G) * U
 *   dU = dA * act(G),  dG = dA * U * act'(G)
 *   dX = dG Wg + dU Wu + scale (dG L2[0]^T) L1[0]^T + scale (dU L2[1]^T) L1[1]^T
 *   dL1[i], dL2[i]: those of qlora_linear_bwd for the upstream gradient dG (i = 0) or dU (i = 1)
 * act(g) = g sigmoid(g) (SILU) or g sigmoid(z), z = sqrt(8 / pi) (g + 0.044715 g^3) (GELU_TANH). G and U are fp32
 * sums of bf16 products (scale T rounded to bf16 before its second product, as in qlora_linear_fwd) and are not
 * rounded before A; dG, dU and scale (dG L2^T), scale (dU L2^T) are rounded to bf16 once, as the operands of the products
 * that follow. A forward call of a single row that keeps no gate8 and up8, of rank up to 64 and K a multiple of 256 with
 * both weights double-quantised in one data type, may take the code values rounded to fp16, which can move a weight to
 * the neighbouring bf16: its A then differs in its last bits from that of a call that keeps them.
 *   gate, up     host structs of the quantised weights, both [F][K] (data types may differ).
 *   X            device bf16 [M][K]; backward: or NULL, with X8 its int8 values (dX, dL1, dL2 are then those of the
 *                values rounded to bf16).
 *   L1, L2       device bf16 [2][K][r], [2][r][F]: gate's adapter, then up's.
 *   A, dA        device bf16 [M][F].
 *   T_out, T     optional device bf16 [2][M][r] = bf16(X L1[i]): written by the forward pass, read by the backward
 *                pass (which computes it when T is NULL).
 *   gate8, up8   optional (both or neither) host structs of the int8 values of G and U (F a multiple of 64): written
 *                by the forward pass; the backward pass takes G and U from them, and without them computes both again
 *                from X.
 *   dX           device bf16 [M][K], or NULL to skip it.
 *   dL1, dL2     device, grad_dtype, shaped like L1, L2.
 *   ws           qlora_gated_workspace(M, K, F, r, backward) bytes.
 * Sums run in a fixed order. An infinity or NaN of one row of X, dA, T or the int8 values reaches no other row of A or
 * dX; through kept values it reaches all 64 features of its block. Both adapters have one rank; there is no adapter
 * dropout. Shapes: K a multiple of 64, F and r of 8, r in [8, 256], K and F below QLORA_GATED_MAX_COLS. M <= 128 in the
 * forward pass streams both 4-bit weights once; a larger M and the backward pass dequantise them into ws.
 */
int qlora_gated_workspace(int64_t M, int64_t K, int64_t F, int r, int backward, size_t *bytes);
int qlora_gated_fwd(const qlora_nf4 *gate, const qlora_nf4 *up, const uint16_t *X, int64_t M, const uint16_t *L1,
                    const uint16_t *L2, int r, float scale, qlora_act act, uint16_t *A, uint16_t *T_out,
                    const qlora_int8_values *gate8, const qlora_int8_values *up8, void *ws, size_t ws_bytes,
                    hipStream_t stream);
int qlora_gated_bwd(const qlora_nf4 *gate, const qlora_nf4 *up, const uint16_t *X, const qlora_int8_values *X8,
                    const uint16_t *dA, int64_t M, const uint16_t *L1, const uint16_t *L2, int r, float scale,
                    qlora_act act, const uint16_t *T, const qlora_int8_values *gate8, const qlora_int8_values *up8,
                    uint16_t *dX, void *dL1, void *dL2, qlora_dtype grad_dtype, void *ws, size_t ws_bytes,
                    hipStream_t stream);

/*
 * qlora_linear_bwd with X as int8 values [M][K]: dL1, and T where it is NULL, come from those values rounded to bf16;
 * dX does not depend on X. There is no adapter dropout (qlora_linear_bwd_dropout has it, from bf16). Arguments otherwise
 * as there, K and N below QLORA_GATED_MAX_COLS; ws: qlora_linear_bwd_int8_workspace(M, K, N, r) bytes.
 */
int qlora_linear_bwd_int8_workspace(int64_t M, int64_t K, int64_t N, int r, size_t *bytes);
int qlora_linear_bwd_int8(const qlora_nf4 *W, const qlora_int8_values *X8, const uint16_t *dY, int64_t M,
                          const uint16_t *L1, const uint16_t *L2, int r, float scale, const uint16_t *T, uint16_t *dX,
                          void *dL1, void *dL2, qlora_dtype grad_dtype, void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * qlora_norm_fwd: h = x + residual, rstd = 1 / sqrt(mean_k h^2 + eps), y = h * rstd * weight, row by row.
 *   x          device, x_dtype, [M][K].
 *   residual   device, stream_dtype, [M][K], or NULL (h = x; stream_dtype is then not used).
 *   weight     device, weight_dtype, [K], or NULL for ones.
 *   y          device bf16 [M][K], or NULL.
 *   y8         host struct of the int8 values of y (K a multiple of 64), or NULL.
 *   h          device, stream_dtype, [M][K]; may be residual itself, or x where the types agree. Given exactly with a
 *              residual.
 *   rstd       device fp32 [M], or NULL.
 * y and its int8 values come from the unrounded h; every output is rounded once.
 *
 * qlora_norm_bwd: with xh = h * rstd,
 *   dh = rstd * (weight * dy - xh * mean_k(weight * dy * xh)) + dres,  dweight = sum over the rows of dy * xh
 *   dy         device bf16 [M][K].
 *   h          device, stream_dtype, [M][K]: the forward pass's h (its x without a residual).  rstd: its rstd.
 *   dres       device, stream_dtype, [M][K]: the gradient that reaches h past the norm, or NULL.
 *   dh         device, stream_dtype, [M][K]: the gradient of x and of residual; may be dres itself.
 *   dx16       device bf16 [M][K]: dh rounded to bf16 (beside an fp32 stream), or NULL.
 *   dweight    device fp32 [K], or NULL.  ws: qlora_norm_workspace(M, K) bytes, needed for dweight only.
 * Sums are fp32 in a fixed order. K: a multiple of 8 up to QLORA_NORM_MAX_COLS.
 */
int qlora_norm_workspace(int64_t M, int64_t K, size_t *bytes);
int qlora_norm_fwd(const void *x, qlora_dtype x_dtype, const void *residual, qlora_dtype stream_dtype,
                   const void *weight, qlora_dtype weight_dtype, int64_t M, int64_t K, float eps, uint16_t *y,
                   const qlora_int8_values *y8, void *h, float *rstd, hipStream_t stream);
int qlora_norm_bwd(const uint16_t *dy, const void *h, qlora_dtype stream_dtype, const float *rstd, const void *weight,
                   qlora_dtype weight_dtype, const void *dres, int64_t M, int64_t K, void *dh, uint16_t *dx16,
                   float *dweight, void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * qlora_head_loss: with the logits S = H W^T, which are not stored,
 *   nll[m] = log sum_v exp(S[m][v]) - S[m][y],  y = labels[m]
 *   loss   = sum over the counted rows of weights[m] nll[m] / divisor
 *   dH     = grad_scale d loss / d H,  dW = grad_scale d loss / d W
 * A row counts when its label lies in [0, V); the others' hidden states are not used, their nll is 0 and their rows of
 * dH are zeros.
 *   H        device bf16 [M][K].   W  device bf16 [V][K].   labels  device int64 [M].
 *   weights  device fp32 [M], or NULL for ones.
 *   divisor  0: the number of counted rows; else the divisor itself (finite, positive).
 *   loss     device fp32 [1] (0 without counted rows).   nll  device fp32 [M].
 *   dH       device bf16 [M][K], or NULL.   dW  device, grad_dtype, [V][K], or NULL.
 *   ws       qlora_head_workspace(M, K, V, dH, dW, grad_dtype) bytes (dH, dW: whether they are computed).
 * Logits and their sums are fp32, the loss is summed in fp64, sums run in a fixed order. The probabilities are rounded
 * to bf16 once as an operand of the gradients' products (twice in rows where a logit is more than 40 above the label's
 * and the vocabulary's tiles are brought to one maximum; for dW, scaled rows of H are rounded too). An infinity or NaN
 * in one row of H reaches no other row of nll or dH.
 * K: a multiple of 64, below 2^23; V in [1, QLORA_HEAD_MAX_VOCAB]. Rows are taken in pieces of at most 2^29 / V (at
 * least 256): the workspace holds the probabilities of one piece, 1 GiB or 512 V bytes at most; none without dH and dW.
 */
int qlora_head_workspace(int64_t M, int64_t K, int64_t V, int dH, int dW, qlora_dtype grad_dtype, size_t *bytes);
int qlora_head_loss(const uint16_t *H, const uint16_t *W, const int64_t *labels, const float *weights, int64_t M,
                    int64_t K, int64_t V, float divisor, float grad_scale, float *loss, float *nll, uint16_t *dH,
                    void *dW, qlora_dtype grad_dtype, void *ws, size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_LAYERS_H */
