/*
 * rms_norm.h -- the root-mean-square norm of a residual stream, with the
 * residual's addition, an output in the rows' type, in 8 bits or in 4 bits,
 * and its gradient, on one GB300 (part of libsgemm_gb300.so; status codes as
 * in sgemm.h, row types as in int8_gemm.h, 4-bit formats as in fp4_gemm.h).
 *
 * For each of M rows of H values:
 *
 *   s   = x + res                 rounded to the row type, and kept in `sum`
 *   rho = 1 / sqrt(mean_h s_h^2 + eps)          (of the rounded s)
 *   y_h = s_h rho weight_h
 *
 * In few bits the row v_h = s_h weight_h is quantised, without rho, and the
 * row's scale carries it: codes and block scales do not hang on the last bits
 * of a sum.
 *   8 bits   as sgemm_i8_quantize_rows(v), scale times rho: the operand A of
 *            sgemm_i8
 *   4 bits   as sgemm_fp4_quantize_rows(v), scale times rho: the operand A of
 *            sgemm_fp4
 *
 * The way back, from dy and the gradient dsum that reaches s by the stream
 * itself (its other users):
 *
 *   m    = mean_h weight_h dy_h s_h
 *   dx   = dsum + rho (weight dy - s rho^2 m)     (for x and res alike)
 *   dweight_h = sum over the rows of dy_h s_h rho
 *
 * Matrices are row-major with leading dimensions in elements (>= H); weight
 * has H values of the row type, dweight H fp32 values.  Every pointer is a
 * DEVICE pointer owned by the caller.  Any alignment of rows to their type is
 * accepted; rows on 16-byte boundaries are fastest.  res, sum, weight (ones),
 * dsum (zeros) and dweight (not wanted) may be NULL.  An output may be one of
 * the inputs of the same shape at the same address and with the same leading
 * dimension (sum and y: x or res; dx: dy or dsum); otherwise outputs may not
 * overlap inputs or each other.
 *
 * Arithmetic: fp32, one rounding to the row type; the sum of squares is held
 * in fp32, and where it leaves fp32's range (4096 values of 2^58) rho is 0: y
 * is zeros, dx is dsum, and the row adds nothing to dweight.  dweight's sums
 * run in an order fixed by the sizes and the alignment: repeated calls give the
 * same bits.  eps must be a normal positive fp32 number.
 *
 * Errors: SGEMM_ERR_INVALID_ARG (dimensions, leading dimensions, type, eps,
 * NULL where data is read or written, misaligned pointers, a workspace that is
 * too small) before anything is launched; SGEMM_ERR_UNSUPPORTED without a
 * compute capability 10.3 GPU; SGEMM_ERR_LAUNCH if a launch fails.  Calls
 * enqueue on `stream` and return; nothing is allocated or synchronised.
 * M == 0: nothing but a zero dweight.  H == 0: nothing but zero scales.
 */
#ifndef RMS_NORM_GB300_H
#define RMS_NORM_GB300_H

#include <stddef.h>

#include "fp4_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* sum (M x H; NULL: not kept) and y (M x H). */
int sgemm_rms_norm(int type, int M, int H, float eps, const void *x, int ldx, const void *res,
                   int ldr, const void *weight, void *sum, int lds, void *y, int ldy,
                   void *stream);

/* sum, and the normed row as 8-bit codes q (M x H, ldq >= H) with one scale
 * (M).  A row with v below 2^-100 throughout gets scale 0 and codes 0, one that
 * holds an infinity or NaN scale NaN and codes 0. */
int sgemm_rms_norm_i8(int type, int M, int H, float eps, const void *x, int ldx, const void *res,
                      int ldr, const void *weight, void *sum, int lds, signed char *q, int ldq,
                      float *scale, void *stream);

/* sum, and the normed row in 4 bits: codes q, block scales sf and row scales,
 * laid out as sgemm_fp4_quantize_rows writes them. */
int sgemm_rms_norm_fp4(int type, int format, int M, int H, float eps, const void *x, int ldx,
                       const void *res, int ldr, const void *weight, void *sum, int lds,
                       unsigned char *q, int ldq, unsigned char *sf, float *scale, void *stream);

/* Bytes of workspace that sgemm_rms_norm_grad needs (0 for invalid
 * dimensions): one fp32 row for each of up to 608 groups of rows.  A call does
 * not read what it did not write there; calls that may run at the same time
 * need one each. */
size_t sgemm_rms_norm_grad_workspace_size(int M, int H);

/* dx (M x H) and dweight (H) from the sum s that the forward call kept and
 * the gradients dy and dsum (M x H).  workspace: 16-byte aligned, not used
 * (and may be NULL) when dweight is NULL. */
int sgemm_rms_norm_grad(int type, int M, int H, float eps, const void *s, int lds,
                        const void *weight, const void *dy, int ldy, const void *dsum, int ldds,
                        void *dx, int ldx, float *dweight, void *workspace,
                        size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* RMS_NORM_GB300_H */
