/*
 * mxmoe.h -- C ABI of the routed-experts operators of libmxfp8.so and of its
 * FP8 products with blocks of 128, on MI355X (gfx950).
 *
 *   mx_route / mx_route_bwd         expert scores, the choice of top experts and
 *       their weights; the gradient of the logits
 *   mx_dispatch                     the choice -> group sizes, offsets and the
 *       two maps between (token, choice) slots and rows in expert order
 *   mx_gather_quantize / mx_b128_gather_quantize   token rows into expert order,
 *       quantized on the way (MXFP8 / blocks of 128), by a weight each if given
 *   mx_combine / mx_combine_bwd     weighted sum of a token's expert rows; the
 *       gradient of the weights
 *   mx_b128_quantize, mx_b128_quantize_weight, mx_b128_mm,
 *   mx_b128_grouped_mm, mx_b128_grouped_mm_wgrad   FP8 with float32 scales of
 *       1 x 128 (activations, gradients) and 128 x 128 (weights)
 *
 * The conventions of mxfp8.h hold (device pointers, row-major tensors, streams,
 * alignment, errors, no allocation, no synchronization). Float32 arrays are
 * 4-byte aligned unless stated, row strides of bf16 matrices at most 2^26 elements,
 * numbers of rows and capacities below 2^31 - 2^16 where no other bound is given.
 * Results do not change from run to run.
 *
 * A "slot" is a token's j-th choice: slot t * top + j.
 *
 * Blocks of 128 ("B128"). Scale of a block with largest magnitude m:
 *   MX_B128_F32    s = float32(max(m, 2^-100) / 448)
 *   MX_B128_RCEIL  the smallest power of two that is not below that
 * codes: E4M3 of float32(v / s), both roundings to nearest even. A block that
 * holds a NaN or infinity gets scale NaN and codes 0x7F with each element's sign.
 * Scales of 1 x 128 blocks of a matrix [R, C] (C a multiple of 128) are stored
 * by block: float32 [C/128, R]; of 128 x 128 blocks float32
 * [ceil(C/128), ceil(R/128)] (an edge block holds what is left).
 */
#ifndef MXMOE_H
#define MXMOE_H

#include "mxfp8.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MX_SOFTMAX = 0, MX_SIGMOID = 1 } mx_score;
typedef enum { MX_GROUP_MAX = 0, MX_GROUP_TOP2 = 1 } mx_group_score;
typedef enum { MX_B128_F32 = 0, MX_B128_RCEIL = 1 } mx_b128_mode;

/* Routing. x: logits [rows, experts] of x_dtype (MX_BF16 or MX_F32), row stride
 * ld >= experts, aligned to its element.
 *   s = float32(softmax(x)) or float32(sigmoid(x)), rounded once from float64 values
 *       off by some 2^-50: the nearest float32 but for about one score in 2^25
 *   c = float32(s + bias)            (c = s if bias is NULL; float32 [experts])
 * An expert whose logit or c is -infinity is ruled out. With groups > 1 the
 * experts form that many groups of equal size in order; a group's value is its
 * largest c (MX_GROUP_MAX) or the float32 sum of its two largest (MX_GROUP_TOP2;
 * one, where one is left), and only the top_groups groups of largest value stay.
 * The `top` experts of largest c are chosen, in descending order. Ties, of groups
 * too, go to the lower index; a NaN counts as larger than any number.
 *   weights float32 [rows, top]: s of the chosen * scale, divided by their sum
 *           if renorm (a sum of 0 divides by 1)
 *   idx     int32 [rows, top]
 * Where fewer than `top` experts are left, the rest has idx -1 and weight 0. A
 * NaN or +infinity among softmax's logits makes its row's weights NaN.
 * 1 <= experts <= 1024, 1 <= top <= min(16, experts), 1 <= groups <= 16 and a
 * divisor of experts, 1 <= top_groups <= groups; rows <= 2^23. */
mx_status mx_route(const void* x, mx_dtype x_dtype, int64_t ld, int64_t rows,
                   int32_t experts, const float* bias, mx_score score,
                   int32_t groups, int32_t top_groups,
                   mx_group_score group_score, int32_t top, int renorm,
                   float scale, float* weights, int32_t* idx, void* stream);

/* Gradient of mx_route's weights with respect to x (the choice and the bias
 * have none): dlogits [rows, experts] of x_dtype, contiguous. idx is the
 * forward's; an entry outside [0, experts) has no part, nor has one whose score is 0
 * as a float32 (a sigmoid's logit below about -104): its weight is 0 whatever the logit, and
 * a row of such scores only gets zeros. */
mx_status mx_route_bwd(const void* x, mx_dtype x_dtype, int64_t ld, int64_t rows,
                       int32_t experts, mx_score score, const int32_t* idx,
                       int32_t top, int renorm, float scale,
                       const float* dweights, void* dlogits, void* stream);

/* int32 elements of the work area of mx_dispatch (0: none needed). */
int64_t mx_dispatch_work(int64_t slots, int32_t experts);

/* Rows in expert order. idx: int32 [slots]; a slot whose entry is outside
 * [0, experts) gets no row. Expert e's rows are its slots in ascending order,
 * its group padded to a multiple of `multiple` rows. Outputs, int32:
 *   sizes [experts]  slots of an expert
 *   offs  [experts]  exclusive ends of the padded groups (as the grouped GEMMs take)
 *   src   [cap]      slot of each row, -1 for padding and behind the last group
 *   pos   [slots]    row of each slot, or -1
 * cap >= slots + min(experts, slots) * (multiple - 1), so that every choice fits;
 * 1 <= experts <= 1024, 1 <= multiple <= 1024, slots and cap below 2^31 - 2^16.
 * work: mx_dispatch_work(slots, experts) elements. */
mx_status mx_dispatch(const int32_t* idx, int64_t slots, int32_t experts,
                      int32_t multiple, int64_t cap, int32_t* sizes,
                      int32_t* offs, int32_t* src, int32_t* pos, int32_t* work,
                      void* stream);

/* Rows gathered and quantized: row r is y_r = x[src[r] / top], zeros where
 * src[r] is negative (or the row is past x), or with weights (float32, by slot)
 * bf16(weights[src[r]] * x[src[r] / top]). x: bf16 [x_rows, cols], row stride ld.
 * q_row [rows, cols], s_row: MX(y) along cols; q_col [cols, rows_pad], s_col:
 * along the rows, filled up with zero rows to rows_pad, the next multiple of the
 * layout's step (both or neither). cols a positive multiple of 128 (32 for
 * MX_SCALES_PLAIN), at most 2^20; rows at most 2^25, rows * cols 2^33; top >= 1. */
mx_status mx_gather_quantize(const void* x, int64_t ld, int64_t x_rows,
                             int64_t cols, const int32_t* src, int32_t top,
                             const float* weights, int64_t rows,
                             mx_scale_mode mode, mx_scale_layout layout,
                             uint8_t* q_row, uint8_t* s_row, uint8_t* q_col,
                             uint8_t* s_col, void* stream);

/* The same in B128: s_row float32 [cols/128, rows], s_col float32
 * [rows_pad/128, cols] with rows_pad a multiple of 128. */
mx_status mx_b128_gather_quantize(const void* x, int64_t ld, int64_t x_rows,
                                  int64_t cols, const int32_t* src, int32_t top,
                                  const float* weights, int64_t rows,
                                  mx_b128_mode mode, uint8_t* q_row, float* s_row,
                                  uint8_t* q_col, float* s_col, void* stream);

/* out_t = bf16(r_t + sum_j w_tj * y[pos_tj]), float32 sums in the order of j:
 * y bf16 [y_rows, cols], row stride ld_y; pos int32 [rows, top], an entry outside
 * [0, y_rows) has no part; weights float32 [rows, top], NULL for ones (the
 * gradient of the gathered rows: the sum of their copies); r bf16 [rows, cols],
 * row stride ld_r, or NULL. out bf16 [rows, cols]. cols a multiple of 8, at most
 * 2^20; rows at most 2^23, rows * cols 2^33; 1 <= top <= 1024. */
mx_status mx_combine(const void* y, int64_t ld_y, int64_t y_rows,
                     const int32_t* pos, const float* weights, const void* r,
                     int64_t ld_r, int64_t rows, int32_t top, int64_t cols,
                     void* out, void* stream);

/* Gradient of the weights of mx_combine: dweights_tj = <dout_t, y[pos_tj]>
 * (float32 [rows, top]), 0 where pos is outside. The gradient of y is
 * mx_gather_quantize of dout with the weights. */
mx_status mx_combine_bwd(const void* dout, int64_t ld_dout, const void* y,
                         int64_t ld_y, int64_t y_rows, const int32_t* pos,
                         int64_t rows, int32_t top, int64_t cols,
                         float* dweights, void* stream);

/* B128 of x, bf16 [rows, cols] (row stride ld), in blocks of 1 x 128: either
 * pair of outputs, along cols (q_row, s_row) and along the rows (q_col, s_col,
 * as above), may be NULL, not both. cols and rows as above. */
mx_status mx_b128_quantize(const void* x, int64_t ld, int64_t rows, int64_t cols,
                           mx_b128_mode mode, uint8_t* q_row, float* s_row,
                           uint8_t* q_col, float* s_col, void* stream);

/* B128 of weights, bf16 [batch, rows, cols], in blocks of 128 x 128: q [batch,
 * rows, cols], s; and, unless q_t is NULL, the transposed copies q_t [batch,
 * cols, rows], s_t (the same numbers). rows, cols multiples of 16, at most 2^24; at most
 * 2^22 blocks in all. */
mx_status mx_b128_quantize_weight(const void* w, int64_t batch, int64_t rows,
                                  int64_t cols, mx_b128_mode mode, uint8_t* q,
                                  float* s, uint8_t* q_t, float* s_t,
                                  void* stream);

/* C = A B^T: A codes [M, K] with scales [K/128, M]; B codes [N, K] with scales
 * [K/128, N] (block_b = 0) or [K/128, ceil(N/128)] (block_b = 1). C [M, N] of
 * out_dtype, row stride ldo elements (rows 16-byte aligned). K a multiple of 128
 * (K = 0 gives zeros), N of 8. Any M; few rows take a kernel that streams B.
 * Here and below a row of codes is shorter than 2^23, one matrix's scales are fewer
 * than 2^29, and a launch takes fewer than 2^22 tiles of 256 x 256 results a group
 * (64 x 128 in grouped products of fewer than 128 rows a group). The matrix unit
 * holds a group of 8 products to 2^-13 of its largest: float32 results are off by some
 * 1.5e-5 of their size. The scales of the two sides are multiplied in float32. */
mx_status mx_b128_mm(const uint8_t* qa, const float* sa, const uint8_t* qb,
                     const float* sb, int block_b, int64_t M, int64_t N,
                     int64_t K, mx_dtype out_dtype, void* out, int64_t ldo,
                     void* stream);

/* Grouped C = A B_g^T for the rows of each group g (forward and input
 * gradient): A codes [cap, K], scales [K/128, cap]; B codes [E, N, K], scales
 * [E, K/128, ceil(N/128)]; offs int32 [E], the groups' ends, of any alignment. C
 * bf16 [cap, N]; rows behind the last group are zeros. Ends that fall or lie
 * outside [0, cap] set bit 0 of *dev_err (if non-NULL); every access stays in
 * bounds. 1 <= E <= 1024; K a positive multiple of 128, N a multiple of 8. */
mx_status mx_b128_grouped_mm(const uint8_t* qa, const float* sa,
                             const uint8_t* qw, const float* sw,
                             const int32_t* offs, int32_t E, int64_t cap,
                             int64_t N, int64_t K, void* out, int32_t* dev_err,
                             void* stream);

/* Weight gradient: dW[g] = G[:, rows of g] X[:, rows of g]^T, out_dtype
 * [E, N, K]: G codes [N, cap], scales [cap/128, N]; X codes [K, cap], scales
 * [cap/128, K]. cap and the ends multiples of 128 (others are reported as above);
 * a group without rows gets zeros. N any, K a multiple of 8. */
mx_status mx_b128_grouped_mm_wgrad(const uint8_t* qg, const float* sg,
                                   const uint8_t* qx, const float* sx,
                                   const int32_t* offs, int32_t E, int64_t cap,
                                   int64_t N, int64_t K, mx_dtype out_dtype,
                                   void* out, int32_t* dev_err, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXMOE_H */
