/*
 * fk_q8.h -- C ABI of libfk, continued: the 8-bit linear layer (sm_100a).
 *
 * The Linear step between the LayerNorm / RMSNorm and the GELU of a
 * transformer block, with its operands in 8 bits, and the two operators that
 * bring activations to 8 bits on the way:
 *
 *   fk_rmsnorm_rows       residual addition + root-mean-square norm, the
 *                         result in the input's type or in 8 bits with one
 *                         scale per row; fk_rmsnorm_rows_bwd its gradients
 *   fk_quantize_rows      rows to 8 bits with one scale each, optionally
 *                         through GELU
 *   fk_matmul_q8          C = act(A B^T * a_scale * b_scale + bias) on the
 *                         tensor cores
 *
 * One operator's output is the next one's input:
 *   rmsnorm (8 bits) -> matmul_q8 -> quantize_rows (GELU) -> matmul_q8.
 *
 * fk.h's conventions on memory, streams, errors, devices and threads hold
 * here too.  Workspace: fk_rmsnorm_rows_bwd (when dgamma is asked for, and for
 * rows that are read value by value, see there) and fk_matmul_q8 (when k is
 * not a multiple of 16, or a or b is not 16-byte aligned: up to (m + n) rows of
 * k codes) take theirs stream-ordered from the library's private pool.  The
 * pool keeps 64 MiB; a larger workspace is mapped anew after each
 * synchronisation, and better given by the caller: the _ws forms take the
 * caller's and allocate nothing.
 *
 * Eight-bit rows.  A row v of fp32 values becomes codes and one fp32 scale:
 *     scale = max(max_j |v_j|, 2^-100) / Q,   code_j = round(v_j / scale),
 * Q = 127 (FK_I8, symmetric: -128 never appears) or 448 (FK_E4M3), rounding
 * to nearest even; the value a code stands for is code * scale.  A row of
 * zeros has codes 0.  A row holding a NaN or an infinity has the scale NaN
 * and codes 0, so everything computed from it is NaN.  In fp32: the scale is
 * the product of the maximum and 1 / Q rounded, v_j / scale the quotient
 * rounded, and that is rounded to the code: scales and codes of given values
 * are those of torch's v.abs().amax(-1) / Q and v / scale on the GPU.  (Rows whose largest magnitude is past
 * 2^110 aside, where the quotient's last bit may differ.)
 */
#ifndef FK_Q8_H
#define FK_Q8_H

#include "fk.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 8-bit storage types (accepted where stated; the other entry points answer
 * FK_ERR_UNSUPPORTED_DTYPE).  Values continue those of fk_dtype. */
typedef enum fk_q8type {
    FK_I8 = 2,  /* signed 8-bit integer */
    FK_E4M3 = 3 /* 8-bit float, 4 exponent and 3 fraction bits, largest value 448, no infinities */
} fk_q8type;

/*
 * fk_rmsnorm_rows -- residual addition and root-mean-square norm over each
 * row of a row-major [rows, cols] matrix, in one pass over HBM:
 *     h_j = x_j + residual_j  (fp32 addition, rounded to `dtype`; h = x
 *                              when residual is NULL),
 *     v_j = h_j / sqrt(sum_i h_i^2 / cols + eps) * gamma_j,
 *     y   = v rounded to `dtype`, or its 8-bit codes and scale.
 *   x         [in]  rows*cols values of `dtype` (FK_F32 or FK_BF16).
 *   residual  [in]  the same shape and type, or NULL.
 *   gamma     [in]  cols fp32 values, or NULL (1).
 *   y         [out] rows*cols values of `out_dtype`: `dtype`, FK_I8 or FK_E4M3.
 *   scales    [out] rows fp32 scales when out_dtype is 8-bit; NULL otherwise.
 *   h         [out] the sum, rows*cols values of `dtype`; NULL = not stored.
 *             Only with a residual.
 *   eps       finite, >= 0.
 * In place: h == x, h == residual (the residual stream updated where it
 * stands), and y == x or y == residual when out_dtype == dtype and h is
 * elsewhere.  Every other overlap of an output with an input or another
 * output is rejected.
 * Arithmetic in fp32.  The row is read once up to 131072 columns; longer rows
 * are read twice, value by value, as are rows of buffers that lie differently:
 * x, residual, h (and y in the rows' type) at different offsets from a 16-byte
 * boundary, or gamma off one.  A row whose h holds a NaN or an infinity, or whose sum of
 * squares overflows fp32 (|h| past about 1e19), is NaN throughout (8-bit:
 * scale NaN, codes 0).  eps == 0 makes a row of zeros NaN, and a row of
 * values whose squares underflow (below about 1e-22) counts as one.  The
 * products h_j gamma_j have to lie within fp32's range.
 * Errors: FK_ERR_INVALID_ARG for bad pointers, overlap, eps, scales present
 * or absent against out_dtype, or h without residual;
 * FK_ERR_UNSUPPORTED_DTYPE for another dtype or out_dtype.
 */
FK_API fk_status fk_rmsnorm_rows(const void *x, const void *residual, const float *gamma, void *y, float *scales,
                                 void *h, size_t rows, size_t cols, int dtype, int out_dtype, float eps,
                                 void *stream);

/*
 * fk_rmsnorm_rows_bwd -- gradients of y = h / sqrt(mean(h^2) + eps) * gamma
 * (fk_rmsnorm_rows with out_dtype == dtype), h = x + residual:
 *     r = 1 / sqrt(sum_i h_i^2 / cols + eps),  s = sum_i dy_i gamma_i h_i / cols,
 *     dx_j     = r dy_j gamma_j - r^3 s h_j  (+ dres_j),
 *     dgamma_j = sum_rows dy_j h_j r.
 * dx is the gradient of x and of residual alike.
 *   dy     [in]  rows*cols values of `dtype` (FK_F32 or FK_BF16).
 *   h      [in]  what was normalised: fk_rmsnorm_rows's h, or its x without
 *                a residual.
 *   gamma  [in]  cols fp32 values, or NULL (1).
 *   dres   [in]  gradient that arrives at h from the residual stream,
 *                rows*cols values of `dtype`, or NULL.
 *   dx     [out] rows*cols values of `dtype`; may be dy, h or dres (in place).
 *   dgamma [out] cols fp32 values, or NULL (not computed).  rows == 0 gives 0.
 *   eps    as in the forward call.
 * The products dy_j gamma_j h_j and their sum over a row have to lie within
 * fp32's range.
 * Arithmetic in fp32; dgamma is summed in fp32 in an order fixed by the
 * shape and the way the buffers lie (two equal calls give equal bits).  Rows
 * up to 65536 columns are read once.  Longer ones, and rows of buffers that lie
 * differently (dy, h, dres and dx at different offsets from a 16-byte boundary,
 * or gamma off one), are read value by value, dy and h three times.
 * Errors as fk_rmsnorm_rows; dgamma must overlap nothing.
 */
FK_API fk_status fk_rmsnorm_rows_bwd(const void *dy, const void *h, const float *gamma, const void *dres, void *dx,
                                     float *dgamma, size_t rows, size_t cols, int dtype, float eps, void *stream);

/* Device workspace, in bytes, that fk_rmsnorm_rows_bwd of this shape uses
 * (want_dgamma: whether dgamma is not NULL).  Host only, no device needed. */
FK_API fk_status fk_rmsnorm_rows_bwd_workspace(size_t rows, size_t cols, int dtype, int want_dgamma, size_t *bytes);

/* fk_rmsnorm_rows_bwd with the caller's workspace (16-byte aligned device
 * memory, at least that many bytes, overlapping nothing else; NULL when that
 * size is 0): allocates nothing.  It must not be used by other work until
 * the call's kernels have finished. */
FK_API fk_status fk_rmsnorm_rows_bwd_ws(const void *dy, const void *h, const float *gamma, const void *dres,
                                        void *dx, float *dgamma, size_t rows, size_t cols, int dtype, float eps,
                                        void *workspace, size_t workspace_bytes, void *stream);

/*
 * fk_quantize_rows -- each row of a row-major [rows, cols] matrix to 8 bits
 * with one scale: v = act(x), codes and scale as above.
 *   x         [in]  rows*cols values of `dtype` (FK_F32 or FK_BF16).
 *   q         [out] rows*cols codes of `out_dtype` (FK_I8 or FK_E4M3); must
 *             not overlap x.
 *   scales    [out] rows fp32 scales; must overlap neither.
 *   epilogue  an fk_epilogue: the values are quantised as they are, or
 *             through GELU in either form (computed in fp32, with the
 *             accuracy of fk_gelu on FK_F32, and of negative values within
 *             2^-14 relative as far down as a code of theirs is not 0).
 * The row is read once up to 131072 columns, twice beyond.
 * Weights [n, k] become per-channel scales by the same call.
 */
FK_API fk_status fk_quantize_rows(const void *x, void *q, float *scales, size_t rows, size_t cols, int dtype,
                                  int out_dtype, int epilogue, void *stream);

/*
 * fk_matmul_q8 -- product of 8-bit matrices with a scale for each row of A
 * (token) and each row of B (output channel):
 *     C[i, j] = act( (sum_l A[i, l] B[j, l]) * a_scales[i] * b_scales[j] + bias[j] )
 *   a         [in]  m*k codes of `dtype`, row-major [m, k].
 *   b         [in]  n*k codes of `dtype`, row-major [n, k] (a Linear weight:
 *             one row per output channel).
 *   a_scales  [in]  m fp32 values.      b_scales [in]  n fp32 values.
 *   bias      [in]  n fp32 values, or NULL.
 *   c         [out] m*n values of `out_dtype` (FK_F32 or FK_BF16), row-major
 *             [m, n]; must overlap no input.
 *   m, n, k   m == 0 or n == 0 is a no-op; m, n, k at most 2^31 - 256; k > 0, and
 *             for FK_I8 k <= 131071 (the exact 32-bit sum of products of codes
 *             down to -128 cannot overflow).
 *   dtype     FK_I8 (sums exact in 32-bit integers) or FK_E4M3 (sums in fp32
 *             on the tensor cores, within (k / 32 + 8) 2^-22 of the sum of the
 *             products' magnitudes).
 *   epilogue  an fk_epilogue applied to the scaled sum in fp32.
 * The sum is converted to fp32, multiplied by a_scales[i] then b_scales[j],
 * bias added, act applied, and rounded once to `out_dtype`.  Two equal calls
 * give equal bits.  k a multiple of 16 with a and b 16-byte aligned runs
 * without workspace; otherwise a and b are first copied to workspace rows
 * padded with zeros to a multiple of 16, whole 128-byte lines apart.  (k a
 * multiple of 128 is best: other pitches make TMA read across lines.)
 * Errors: FK_ERR_INVALID_ARG for a shape outside the above, bad pointers or
 * overlap; FK_ERR_UNSUPPORTED_DTYPE for another dtype or out_dtype.
 * A wait that gives up inside the kernel (see fk_wait_timeouts; after 1 s, for
 * a finished product 1 s and 2 us for each 128 codes of k) leaves that part of
 * C unwritten.
 */
FK_API fk_status fk_matmul_q8(const void *a, const void *b, const float *a_scales, const float *b_scales,
                              const float *bias, void *c, size_t m, size_t n, size_t k, int dtype, int out_dtype,
                              int epilogue, void *stream);

/* Device workspace, in bytes, that fk_matmul_q8 uses (0 when `aligned`: a
 * and b both on 16-byte boundaries, and k is a multiple of 16).  Host only. */
FK_API fk_status fk_matmul_q8_workspace(size_t m, size_t n, size_t k, int aligned, size_t *bytes);

/* fk_matmul_q8 with the caller's workspace (16-byte aligned, overlapping
 * nothing else; NULL when that size is 0): allocates nothing. */
FK_API fk_status fk_matmul_q8_ws(const void *a, const void *b, const float *a_scales, const float *b_scales,
                                 const float *bias, void *c, size_t m, size_t n, size_t k, int dtype, int out_dtype,
                                 int epilogue, void *workspace, size_t workspace_bytes, void *stream);

/* Self-test of the above: fk_matmul_q8 into fp32 whose waits for the finished
 * product give up at once, each counted in fk_wait_timeouts.  C is left as it
 * is; what runs inside the kernel ends before the kernel does. */
FK_API fk_status fk_matmul_q8_wait_selftest(const void *a, const void *b, const float *a_scales,
                                            const float *b_scales, float *c, size_t m, size_t n, size_t k, int dtype,
                                            void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FK_Q8_H */
