/*
 * gq_step.h -- the two ends of a training step on AMD Instinct MI355X (gfx950).
 *
 * C ABI of libgq_step.so, next to gq_train.h: the products of linear layers in
 * 8-bit floating point, and the update that takes the reduced gradients --
 * AdamW over many tensors at once, its states in 32 or 8 bits, with the
 * gradients' norm and the factor that clips it.
 *
 * e4m3 copies
 *   - A block of values shares a power of two 2^E.  With a the largest |x| of
 *     the block, E is the smallest integer >= -117 with a <= 448 2^E; a value
 *     is kept as the e4m3 number (4 exponent bits, 3 mantissa bits, no
 *     infinities) x 2^-E rounded, and stands for that number times 2^E, which
 *     float and bfloat16 both hold exactly.  The block's byte is E + 127
 *     (10 .. 247).  With E = 120 the numbers go to 240 (256 2^120 has no
 *     float).
 *   - A block that holds an inf or NaN gets the byte 255 and zero codes; all
 *     its values stand for NaN.
 *   - GQS_ROUND_NEAREST: ties to even.  GQS_ROUND_RANDOM: with f the fraction
 *     of the way from the lower neighbour of |x| 2^-E to the upper, up where
 *     u + floor(f 2^16 + 1/2) >= 2^16: unbiased, up to 2^-17 of a step
 *     (between the format's numbers below its least normal one, f is first
 *     rounded to a multiple of 2^-20).  u is 16-bit half c % 8 of the
 *     Philox4x32-10 block at counter (c / 8, 0, row, 0) under the key `seed`,
 *     c the column.
 *   - Rows: a block is 128 columns of a row; codes [rows][128 G] with G =
 *     ceil(d / 128) (columns past d hold 0), exps [G][16 ceil(rows / 16)].
 *   - Weights: w[n][k] has a block for each square of 128 x 128; codes
 *     [n][128 Gk], exps [Gn][Gk], and codes_t [k][128 Gn] the same codes
 *     transposed.
 *
 * Moments in 8 bits
 *   - A tensor of n elements has blocks of 128 elements in order: codes
 *     [128 G] (those past n hold 0) and exps [G], G = ceil(n / 128).
 *   - The first moment: e4m3, as above.  The second: 5 exponent bits and 3
 *     mantissa bits without a sign; c < 8 is c 2^-18, otherwise
 *     (1 + (c & 7) / 8) 2^((c >> 3) - 16).  Its E is the smallest integer >=
 *     -108 with a <= 61440 2^E; with E = 113 the numbers go to 30720.
 *   - They are rounded at random (to nearest, a moment that shrinks by a
 *     thousandth a step would never move): u for element i of the list's
 *     tensor j in step t is half i % 8 of the block at counter (i / 8, t, j,
 *     draw), draw 0 for the first moment, 1 for the second.
 *
 * Conventions shared by every entry point
 *   - Matrices, dtypes, strides, memory, streams, errors and status values as
 *     in gq_train.h; codes and exps are 16-byte aligned.
 *   - Sizes: rows >= 0 and < 2^31, matrix sides in [1, 2^22], rows times
 *     blocks < 2^27.
 *   - No atomics: the same call gives the same bits.
 */
#ifndef GQ_STEP_H
#define GQ_STEP_H

#include <stddef.h>
#include <stdint.h>

#include "gq.h" /* the status values and the dtypes */

#ifdef __cplusplus
extern "C" {
#endif

enum { GQS_ROUND_NEAREST = 0, GQS_ROUND_RANDOM = 1 };

/* G = ceil(d / 128); 128 G, the bytes of a row of codes; -1 for d outside
 * [1, 2^22].  16 ceil(rows / 16), the bytes of a row copy's exps for each
 * block; -1 for rows outside [0, 2^31).                                    */
int64_t gqs_fp8_blocks(int64_t d);
int64_t gqs_fp8_pitch(int64_t d);
int64_t gqs_fp8_exp_pitch(int64_t rows);

/* The row copy of x[rows][d].                                              */
int32_t gqs_fp8_rows(const void *x, int32_t dtype, int64_t rows, int64_t d, int64_t ldx,
                     int32_t rounding, uint64_t seed, void *codes, void *exps, void *stream);

/* The copy of a weight w[n][k], to nearest; codes_t may be NULL.           */
int32_t gqs_fp8_weight(const void *w, int32_t dtype, int64_t n, int64_t k, int64_t ldw,
                       void *codes, void *codes_t, void *exps, void *stream);

/* The values a row copy (squares 0) or a weight's (squares 1) stands for.  */
int32_t gqs_fp8_restore(const void *codes, const void *exps, int64_t rows, int64_t d,
                        int32_t squares, int32_t dtype, void *out, void *stream);

/* y[m][cols] = x w'^T + bias over `depth` columns of x.  transposed 0: w' is
 * the weight [cols][depth] and w_codes its codes; transposed 1: w' is the
 * transpose of the weight [depth][cols] and w_codes its codes_t.  w_exps are
 * the weight's exps either way.  bias [cols] in bias_dtype, or NULL.
 * y in dtype.  fp32 results, and bf16 ones of up to 16 rows, are sums in fp32
 * of exact products, as those of up to 128 rows are where no tile of more is
 * faster.  For other bf16 ones the matrix cores add eight-bit products in
 * groups of eight, of which each of the seven others can lose 2^-13 of the
 * largest: up to 7 2^-13 of it in a group.  The
 * workspace size also depends on m; 0 bytes may come as NULL.              */
int64_t gqs_fp8_product_workspace_bytes(int64_t m, int64_t cols, int64_t depth, int32_t dtype);
int32_t gqs_fp8_product(const void *x_codes, const void *x_exps, int64_t m, const void *w_codes,
                        const void *w_exps, int64_t cols, int64_t depth, int32_t transposed,
                        const void *bias, int32_t bias_dtype, void *y, int32_t dtype,
                        void *workspace, int64_t workspace_bytes, void *stream);

/* The same from x[m][depth] itself: its row copy, rounded as in gqs_fp8_rows,
 * is made on the way.  y has x's dtype.                                    */
int64_t gqs_fp8_linear_workspace_bytes(int64_t m, int64_t cols, int64_t depth, int32_t dtype);
int32_t gqs_fp8_linear(const void *x, int32_t dtype, int64_t m, int64_t depth, int64_t ldx,
                       int32_t rounding, uint64_t seed, const void *w_codes, const void *w_exps,
                       int64_t cols, int32_t transposed, const void *bias, int32_t bias_dtype,
                       void *y, void *workspace, int64_t workspace_bytes, void *stream);

/* A parameter, its gradient and its moments: flat arrays of n elements.
 * With 8-bit moments m and v are their codes, and the exps are read.       */
typedef struct gqs_tensor {
    void *p;
    const void *g;
    void *m;
    void *v;
    void *m_exps;
    void *v_exps;
    int64_t n; /* >= 0, < 2^34 */
} gqs_tensor;

typedef struct gqs_adamw_args {
    double lr, beta1, beta2, eps, weight_decay;
    int64_t step;               /* the number of this step, from 1 */
    const float *scale;         /* device: the gradients' factor, or NULL: 1 */
    const float *lr_device;     /* device: takes lr's place, or NULL */
    const int64_t *step_device; /* device: takes step's place, or NULL */
    uint64_t seed;
    int32_t random; /* whether a bf16 p is rounded at random; 8-bit moments are */
    int32_t bits;   /* 32 or 8 */
} gqs_adamw_args;

/* One step over `count` tensors (a host array), in place:
 *   g' = scale g, m = beta1 m + (1 - beta1) g', v = beta2 v + (1 - beta2) g'^2,
 *   p = p (1 - lr weight_decay)
 *       - lr m / (1 - beta1^step) / (sqrt(v / (1 - beta2^step)) + eps),
 * in fp32; the update takes the moments before their rounding.  With 8-bit
 * moments the first root is that of v or, where that is more, of 2^(E - 18), E
 * the exponent of v's block as it came: the block's lowest step.  Elements of
 * gradients below about 2^-17 of their block's largest keep a v of mostly 0
 * and an m that is 0 or a whole lowest step, whose quotient alone has no bound
 * (300 steps of normal gradients: up to 850 lr where 32-bit moments take 1.3);
 * so their steps were at most 1.8 lr, and shrink with the gradient, as with a
 * larger eps.  Root and quotient are then good to a unit in
 * their last place.  A bf16 p is
 * rounded once, to nearest, or, with `random`, at random: the 16 bits below
 * its last place get the half of draw 2 added.  lr >= 0, 0 <= beta < 1, eps
 * >= 0, step >= 1.  No two tensors may overlap.  The workspace (16 bytes) is
 * needed with lr_device or step_device.                                    */
int32_t gqs_adamw(const gqs_tensor *tensors, int64_t count, int32_t p_dtype, int32_t g_dtype,
                  const gqs_adamw_args *args, void *workspace, int64_t workspace_bytes,
                  void *stream);

/* The values of a moment in 8 bits, first (second 0) or second.            */
int32_t gqs_moment8_restore(const void *codes, const void *exps, int64_t n, int32_t second,
                            int32_t dtype, void *out, void *stream);

/* norm = sqrt(sum over all tensors of g^2), summed in fp64 (of each tensor g
 * and n are read), and, unless NULL, scale = min(1, max_norm / (norm +
 * 1e-6)): device floats.  A NaN among the gradients makes both NaN; an inf
 * gives inf and 0.                                                         */
int64_t gqs_grad_norm_workspace_bytes(const gqs_tensor *tensors, int64_t count);
int32_t gqs_grad_norm(const gqs_tensor *tensors, int64_t count, int32_t dtype, double max_norm,
                      float *norm, float *scale, void *workspace, int64_t workspace_bytes,
                      void *stream);

/* Text of the calling thread's most recent failure in this library.       */
const char *gqs_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* GQ_STEP_H */
