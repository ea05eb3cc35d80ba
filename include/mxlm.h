/*
 * mxlm.h -- C ABI of the layer-boundary operators of libmxfp8.so: what an
 * MXFP8 transformer runs between its GEMMs, on MI355X (gfx950).
 *
 *   mx_add_rmsnorm_quant / mx_add_rmsnorm_bwd   in front of a GEMM: residual
 *       addition, RMS norm and the MXFP8 operand, with an 8-bit checkpoint of
 *       the residual stream; and the gradient
 *   mx_swiglu_ckpt_fwd / mx_swiglu_ckpt_bwd     between two GEMMs: SwiGLU, the
 *       MXFP8 operand, and its input kept for the backward in 8 bits
 *   mx_token_logprobs / mx_token_logprobs_bwd   behind the head GEMM: log
 *       probabilities of given tokens, entropy, top alternatives, and the
 *       gradient of the logits as the MXFP8 operand of the head's two
 *       gradient GEMMs
 *
 * The conventions of mxfp8.h hold (device pointers, row-major tensors, scale
 * layouts, streams, alignment, errors, no allocation, no synchronization),
 * with one addition: the token count T ("rows") may be any number >= 0.
 * Column-wise codes are taken over the rows filled up with zero rows to
 * T_pad, the next multiple of the layout's step (128 for MX_SCALES_K128, 32
 * for MX_SCALES_PLAIN): q_col [cols, T_pad], s_col the scales of that matrix.
 * They are then operands of mx_scaled_mm with K = T_pad. Row strides are at
 * most 2^26 elements where nothing else is stated, and a tensor that is
 * quantized has at most 2^21 tiles of 128 x 128 (2^35 elements).
 *
 * "MX(v)" below is the quantization of mx_quantize in the call's mode and
 * layout, applied to a bf16 matrix.
 */
#ifndef MXLM_H
#define MXLM_H

#include "mxfp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Residual addition + RMS norm + MX quantization.
 *   s    = bf16(x + r)                  (s = x if r is NULL)
 *   rstd = (mean_c s^2 + eps)^(-1/2)    (float32)
 *   y    = bf16((s * rstd) * w)
 * x, r: bf16 [rows, cols], row strides ld_x, ld_r elements; w: float32 [cols],
 * 16-byte aligned. Outputs:
 *   sum    bf16 [rows, cols] = s; required with r, NULL without
 *   rstd   float32 [rows]
 *   q_row, s_row   MX(y) along cols
 *   q_col, s_col   MX(y) along the rows (see T_pad above), or both NULL
 *   q_ck, s_ck     MX(s) along cols: the 8-bit checkpoint, or both NULL
 * cols a positive multiple of 32 (128 for MX_SCALES_K128), at most 16384;
 * eps >= 0. */
mx_status mx_add_rmsnorm_quant(const void* x, int64_t ld_x, const void* r,
                               int64_t ld_r, const float* w, int64_t rows,
                               int64_t cols, float eps, mx_scale_mode mode,
                               mx_scale_layout layout, void* sum, float* rstd,
                               uint8_t* q_row, uint8_t* s_row, uint8_t* q_col,
                               uint8_t* s_col, uint8_t* q_ck, uint8_t* s_ck,
                               void* stream);

/* float32 elements of the work area of mx_add_rmsnorm_bwd. */
int64_t mx_add_rmsnorm_bwd_work(int64_t rows, int64_t cols);

/* Gradient of mx_add_rmsnorm_quant. With xh = s * rstd and g = dy * w:
 *   dx = bf16((g - xh * mean_c(g * xh)) * rstd + dsum)
 *   dw = sum over rows of dy * xh       (float32, fixed order of summation)
 * dx is the gradient of x and of r. dsum: bf16, the gradient that reaches s
 * past the norm (the residual stream), or NULL. s comes from exactly one of
 * x (bf16, the forward's sum, row stride ld_x) and q_ck / s_ck (its
 * checkpoint in the call's layout). Outputs: dx bf16 [rows, cols], dw float32
 * [cols], and MX(dx) along cols (q_row, s_row) and along the rows (q_col,
 * s_col); either pair may be NULL. work: float32 scratch of
 * mx_add_rmsnorm_bwd_work(rows, cols) elements. */
mx_status mx_add_rmsnorm_bwd(const void* dy, int64_t ld_dy, const float* w,
                             const float* rstd, const void* x, int64_t ld_x,
                             const uint8_t* q_ck, const uint8_t* s_ck,
                             const void* dsum, int64_t ld_dsum, int64_t rows,
                             int64_t cols, mx_scale_mode mode,
                             mx_scale_layout layout, void* dx, float* dw,
                             uint8_t* q_row, uint8_t* s_row, uint8_t* q_col,
                             uint8_t* s_col, float* work, void* stream);

/* mx_swiglu_quant_fwd for any number of rows, which also keeps its input in
 * 8 bits: q_row / s_row and q_col / s_col as there (column-wise over T_pad
 * rows), q_ck [rows, 2*hidden] / s_ck = MX([a | b]) along 2*hidden.
 * hidden a positive multiple of 32 (128 for MX_SCALES_K128), at most 2^25. */
mx_status mx_swiglu_ckpt_fwd(const void* a, const void* b, int64_t ld_ab,
                             int64_t rows, int64_t hidden, mx_scale_mode mode,
                             mx_scale_layout layout, uint8_t* q_row,
                             uint8_t* s_row, uint8_t* q_col, uint8_t* s_col,
                             uint8_t* q_ck, uint8_t* s_ck, void* stream);

/* mx_swiglu_quant_bwd with a and b taken from the checkpoint (their values
 * under it): dZ = bf16([dA | dB]) [rows, 2*hidden], MX(dZ) along 2*hidden and
 * along the rows (T_pad). dh: bf16 [rows, hidden], row stride ld_dh. */
mx_status mx_swiglu_ckpt_bwd(const void* dh, int64_t ld_dh, const uint8_t* q_ck,
                             const uint8_t* s_ck, int64_t rows, int64_t hidden,
                             mx_scale_mode mode, mx_scale_layout layout,
                             uint8_t* q_row, uint8_t* s_row, uint8_t* q_col,
                             uint8_t* s_col, void* stream);

/* Bytes of the work area of mx_token_logprobs (0: none needed). */
int64_t mx_token_logprobs_work(int64_t rows, int64_t vocab, int32_t top);

/* Log probabilities of given tokens under softmax(scale * x).
 * x: [rows, vocab] of x_dtype (MX_BF16 or MX_F32), row stride ld >= vocab,
 * aligned to its element only. targets: int64 [rows]; a row whose target is
 * ignore_index is not scored. Outputs, per row, with d_j = (x_j - m) * scale:
 *   stats    float32 [rows, 2]: m = max_j x_j and ls = log sum_j e^(d_j)
 *   logp     float32 [rows]: d_target - ls, 0 where not scored
 *   entropy  float32 [rows]: ls - sum_j p_j d_j
 *   top_logp float32, top_idx int32 [rows, top]: the `top` largest x in
 *            descending order, ties to the lower index (top = 0: both NULL)
 * ls and entropy are never below 0, logp and top_logp never above it. Entries of
 * -infinity are ruled out (p = 0). A row with nothing left has entropy 0,
 * ls = -infinity and logp = -infinity; a NaN or +infinity makes its row's results
 * NaN (top_idx: distinct tokens all the same, those with NaN first).
 * 1 <= vocab < 2^31 - 2^16, 0 <= top <= min(64, vocab); scale in
 * [1e-6, 1e6]. A target outside [0, vocab) that is not ignore_index is
 * treated as not scored and sets bit 3 of *dev_err if that is non-NULL.
 * work: scratch of mx_token_logprobs_work bytes, 16-byte aligned. */
mx_status mx_token_logprobs(const void* x, mx_dtype x_dtype, int64_t ld,
                            int64_t rows, int64_t vocab,
                            const int64_t* targets, int64_t ignore_index,
                            float scale, int32_t top, float* logp,
                            float* entropy, float* stats, float* top_logp,
                            int32_t* top_idx, void* work, int32_t* dev_err,
                            void* stream);

/* Gradient of mx_token_logprobs with respect to x, as an MX operand. With
 * l_j = (x_j - m) * scale - ls and p_j = e^(l_j):
 *   G_j = bf16(scale * (dlogp * ([j = target] - p_j)
 *                       - dent * p_j * (l_j + entropy)))
 * with dlogp taken as 0 in rows that are not scored; dlogp, dent float32
 * [rows], either NULL for zeros; stats and entropy are the forward's. The row
 * is filled up with zeros to V_pad, the next multiple of the layout's step:
 * q_row [rows, V_pad], s_row MX(G) along the vocabulary; q_col
 * [V_pad, T_pad], s_col along the rows. A row with nothing left has gradient
 * 0, and so has an entry that is ruled out, unless it is the target, as long as
 * scale * |dlogp| and 1024 * scale * |dent| stay below 2^100. ld <= 2^26 and vocab <= 2^26 - 128 for bf16, half of that for float32. */
mx_status mx_token_logprobs_bwd(const void* x, mx_dtype x_dtype, int64_t ld,
                                int64_t rows, int64_t vocab,
                                const int64_t* targets, int64_t ignore_index,
                                const float* stats, const float* entropy,
                                const float* dlogp, const float* dent,
                                float scale, mx_scale_mode mode,
                                mx_scale_layout layout, uint8_t* q_row,
                                uint8_t* s_row, uint8_t* q_col, uint8_t* s_col,
                                int32_t* dev_err, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXLM_H */
