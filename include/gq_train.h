/*
 * gq_train.h -- training operators on AMD Instinct MI355X (gfx950).
 *
 * C ABI of libgq_train.so: what a transformer block computes and keeps
 * between its forward and backward passes, next to the gradient compression
 * of gq.h -- layer norm, GELU, activations kept in 8 bits, and the weight
 * gradient of a linear layer taken from the kept codes.
 *
 * The 8-bit copy of a matrix x[rows][d] (gqt_act8)
 *   - The columns of a row fall into groups of 32; G = ceil(d / 32).
 *   - codes: int8 [rows][32 G] (the columns past d hold 0).
 *   - exps: uint8 [rows][G].  With a the largest |x| of the group, E is the
 *     smallest integer >= -126 with a <= 127 2^E, the byte is E + 127
 *     (1 .. 249), and a code q stands for q 2^E, a value that float and
 *     bfloat16 both hold exactly.
 *   - A group that holds an inf or NaN gets the byte 255 and zero codes; all
 *     its values stand for NaN.
 *   - GQT_ROUND_NEAREST: q = x 2^-E to the nearest integer, ties to even.
 *   - GQT_ROUND_RANDOM: |q| = floor(|x| 2^-E) + [u < floor(frac 2^32)] with
 *     the sign of x: unbiased, up to 2^-32 of a step.  u is the 32-bit
 *     uniform gq.h describes (Philox4x32-10, key = seed), with the matrix
 *     row in the place of the worker and the column in the row as the
 *     coordinate.
 *   - |q| <= 127; in a group with E = 122, |q| <= 63 (64 2^122 has no float).
 *
 * Conventions shared by every entry point
 *   - Matrices are row-major.  ld* is the distance between rows in
 *     elements: at least d, or 0 for one row read as every row.  Outputs are
 *     contiguous ([rows][d]).  Matrices and vectors need the alignment of
 *     their element type only, codes 16 bytes.
 *   - dtype: GQ_IN_F32 or GQ_IN_BF16.  Arithmetic and sums are fp32; a
 *     bf16 output is rounded once, to nearest, ties to even.
 *   - Sizes: rows >= 0 and < 2^32, 1 <= d < 2^27, and rows ceil(d / 32)
 *     < 2^29 (17 G values).  rows == 0 enqueues nothing (the sums over rows
 *     are zeros), and the matrices may then be NULL.
 *   - Memory: device pointers owned by the caller.  The library allocates
 *     nothing and keeps no state.  Workspaces need no initialization.
 *   - Streams, errors and status values as in gq.h: calls only enqueue
 *     kernels, every argument check runs before any HIP call, and
 *     gqt_last_error() describes the calling thread's most recent failure.
 *   - No atomics: the same call gives the same bits.
 */
#ifndef GQ_TRAIN_H
#define GQ_TRAIN_H

#include <stddef.h>
#include <stdint.h>

#include "gq.h" /* the status values and the dtypes */

#ifdef __cplusplus
extern "C" {
#endif

enum { GQT_ROUND_NEAREST = 0, GQT_ROUND_RANDOM = 1 };
enum { GQT_GELU_ERF = 0, GQT_GELU_TANH = 1 };

typedef struct gqt_act8 {
    void *codes;      /* int8 [rows][gqt_act8_code_pitch(d)] */
    void *exps;       /* uint8 [rows][gqt_act8_groups(d)] */
    int32_t rounding; /* read where a copy is written */
    uint64_t seed;    /* read with GQT_ROUND_RANDOM */
} gqt_act8;

/* G = ceil(d / 32) and 32 G, the bytes of a row's exps and codes; -1 for
 * d outside [1, 2^27).                                                     */
int64_t gqt_act8_groups(int64_t d);
int64_t gqt_act8_code_pitch(int64_t d);

/* Writes the 8-bit copy of x; out = the values it stands for, in dtype.   */
int32_t gqt_act8_save(const void *x, int32_t dtype, int64_t rows, int64_t d, int64_t ldx,
                      const gqt_act8 *out, void *stream);
int32_t gqt_act8_restore(const gqt_act8 *in, int64_t rows, int64_t d, int32_t dtype, void *out,
                         void *stream);

/* Layer norm of each row:
 *   mean = sum x / d, rstd = 1 / sqrt(sum (x - mean)^2 / d + eps),
 *   y = (x - mean) rstd w + b.
 * y has x's dtype; w and b (each may be NULL: 1 and 0) have wdtype.  mean
 * and rstd (float [rows]) may be NULL.  save_x and save_y, where given,
 * receive the 8-bit copies of x and of the rounded y in the same pass.     */
int32_t gqt_layer_norm(const void *x, int32_t dtype, int64_t rows, int64_t d, int64_t ldx,
                       const void *w, const void *b, int32_t wdtype, float eps, void *y,
                       float *mean, float *rstd, const gqt_act8 *save_x, const gqt_act8 *save_y,
                       void *stream);

/* Its gradient, with xh = (x - mean) rstd and g = dy w:
 *   dx = rstd (g - sum g / d - xh sum(g xh) / d),
 *   dw = sum over rows of dy xh, db = sum over rows of dy.
 * x is given as itself (dtype, ldx) or, with x NULL, as its 8-bit copy x8.
 * dx has dy's dtype (= x's); dw and db (each may be NULL) have wdtype.  The
 * workspace (fp32 partial sums) may be NULL when both are.                 */
int64_t gqt_layer_norm_backward_workspace_bytes(int64_t rows, int64_t d);
int32_t gqt_layer_norm_backward(const void *dy, int32_t dtype, int64_t rows, int64_t d,
                                int64_t lddy, const void *x, int64_t ldx, const gqt_act8 *x8,
                                const float *mean, const float *rstd, const void *w,
                                int32_t wdtype, void *dx, void *dw, void *db, void *workspace,
                                int64_t workspace_bytes, void *stream);

/* GELU, y = h Phi(h) (form GQT_GELU_ERF) or y = h s(2 u) with the logistic
 * function s and u = sqrt(2/pi) (h + 0.044715 h^3) (GQT_GELU_TANH).  save_h
 * and save_y receive 8-bit copies as in gqt_layer_norm.                    */
int32_t gqt_gelu(const void *h, int32_t dtype, int64_t rows, int64_t d, int64_t ldh, int32_t form,
                 void *y, const gqt_act8 *save_h, const gqt_act8 *save_y, void *stream);

/* dh = dy y'(h), with h given as itself or, with h NULL, as its copy h8.  */
int32_t gqt_gelu_backward(const void *dy, int32_t dtype, int64_t rows, int64_t d, int64_t lddy,
                          const void *h, int64_t ldh, const gqt_act8 *h8, int32_t form, void *dh,
                          void *stream);

/* Gradient of y = x w^T + bias with respect to w[n][k] and bias[n], from
 * dy[m][n] and the 8-bit copy x8 of x[m][k]:
 *   dw = dy^T x, db = sum over rows of dy (may be NULL), both in wdtype.
 * Products are exact (an fp32 dy is taken as the sum of three bf16 parts,
 * which hold it whole from |dy| = 2^-110 on; below, what lies under 2^-133
 * is left out) and the sums are fp32.  n and k lie in [1, 2^27), and
 * n k < 2^36.  With m == 0, dw and db are zeros.  dy: lddy >= n, or 0.     */
int64_t gqt_weight_grad_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t dtype);
int32_t gqt_weight_grad(const void *dy, int32_t dtype, int64_t m, int64_t n, int64_t lddy,
                        const gqt_act8 *x8, int64_t k, void *dw, void *db, int32_t wdtype,
                        void *workspace, int64_t workspace_bytes, void *stream);

/* Text of the calling thread's most recent failure in this library.       */
const char *gqt_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* GQ_TRAIN_H */
