/*
 * fp4_gemm.h -- matrix products in microscaled 4-bit floating point on one
 * GB300 (part of libsgemm_gb300.so; status codes as in sgemm.h, row types and
 * acts as in int8_gemm.h).
 *
 * A value is  code * block scale * row scale:
 *   code         4 bits, sign and e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6
 *   block scale  8 bits, shared by consecutive values of a row:
 *                SGEMM_FP4_MX  32 values, a power of two: 2^(byte - 127)
 *                SGEMM_FP4_NV  16 values, e4m3 (sign bit clear)
 *   row scale    fp32, one per row (NULL: 1 everywhere)
 *
 *   C[m][n] = scaleA[m] * scaleB[n] *
 *             sum_k (A[m][k] sfA[m][k/b]) * (B[n][k] sfB[n][k/b])
 *
 * Layout, the same for activations A (M x K) and weights B (N x K):
 *   codes         row-major, two to a byte, the even k in the low half; ld in
 *                 VALUES, a multiple of 32, >= K; 16-byte aligned base.  With
 *                 odd K the high half of a row's last byte must be zero.
 *   block scales  in tiles of 128 rows by 4 blocks, 512 contiguous bytes, the
 *                 tiles of the same rows side by side (ceil(blocks / 4) of
 *                 them): the scale of row r, block j is at byte
 *                   ((r / 128) * ceil(blocks / 4) + j / 4) * 512
 *                   + (r % 32) * 16 + (r % 128) / 32 * 4 + j % 4,
 *                 as the tensor cores take them; 16-byte aligned base;
 *                 sgemm_fp4_scales_size bytes.  Bytes of blocks past the last
 *                 must not be a NaN (zeros, as the quantiser writes them);
 *                 bytes of rows past the last may be anything.
 * Every pointer is a DEVICE pointer owned by the caller.  Calls enqueue on
 * `stream` and return; nothing is allocated or synchronised.
 *
 * Arithmetic: a product of two codes and their block scales is exact; the
 * sums over k are fp32 on the matrix units, cut, not rounded, near fp32's last
 * place of the largest number added.  The row scales are applied in fp32
 * (token first), the result is rounded once to its type.  The same row may
 * give slightly different results in calls of other sizes.  Block scales that
 * hold a NaN give NaN.
 *
 * Errors: SGEMM_ERR_INVALID_ARG (dimensions, leading dimensions, type, format,
 * NULL where data is read or written, misaligned pointers) before anything is
 * launched; SGEMM_ERR_UNSUPPORTED without a compute capability 10.3 GPU;
 * SGEMM_ERR_LAUNCH if a launch fails; a bounded wait that runs out is reported
 * by sgemm_poll_error.
 */
#ifndef FP4_GEMM_GB300_H
#define FP4_GEMM_GB300_H

#include <stddef.h>

#include "int8_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SGEMM_FP4_MX 0
#define SGEMM_FP4_NV 1

/* Bytes of the block scales of `rows` rows of K values (0 for invalid
 * arguments). */
size_t sgemm_fp4_scales_size(int format, int rows, int K);

/* Quantises M rows of K values (2 K with SGEMM_ACT_SWIGLU: K gates, then K
 * values, silu(X[r][k]) * X[r][K + k]) of X into codes Q, block scales sf and
 * row scales (M).  ldx >= K (2 K).
 *   MX  a block's scale is 2^(floor(log2 amax) - 2), at least 2^-127; row scale 1
 *   NV  with a_r the row's largest magnitude, row scale a_r / 2688, a block's
 *       scale e4m3(amax * (448 / a_r)) to nearest
 * Codes are the nearest 4-bit value of x times the scales' inverse, in fp32,
 * ties to the even code, 6 beyond 6.
 * The gated activation is held in fp32, each value within 8 units of fp32's last
 * place (gates below -87, whose exponential is subnormal: 2^-141 |X[r][K + k]|
 * besides).
 *  - A zero's code has the value's sign (0 or 8).
 *  - NV: a row whose largest magnitude is below 2^-100 (zeros among them) gets
 *    row scale 0, block scales 0 and codes of zeros; so does a block whose scale
 *    rounds to 0.
 *  - A row that holds an infinity or NaN, or whose gated activation leaves
 *    fp32's range, gets row scale NaN, block scales 0 and codes 0.
 * Codes from K to the next multiple of 8, and block scales from the last block
 * to the next multiple of 4, are written as zeros; nothing else is.  M == 0 or
 * K == 0: nothing but scales: 0 (NV), 1 (MX). */
int sgemm_fp4_quantize_rows(int type, int act, int format, int M, int K, const void *X, int ldx,
                            unsigned char *Q, int ldq, unsigned char *sf, float *scale,
                            void *stream);

/* C (M x N, `type`, ldc >= N) from A and B.  K == 0 writes zeros times the
 * scales.  C may not overlap the inputs.  M and N <= 2^31 - 512,
 * K <= 2^31 - 8192. */
int sgemm_fp4(int type, int format, int M, int N, int K, const unsigned char *A, int lda,
              const unsigned char *sfA, const float *scaleA, const unsigned char *B, int ldb,
              const unsigned char *sfB, const float *scaleB, void *C, int ldc, void *stream);

/* Hooks for tests and measurement.  A product runs on one of four kernels,
 * chosen by a rule on its sizes:
 *   FEW     up to four tokens
 *   NARROW  tensor cores, 128 channels x 128 tokens a CTA; the CTAs of a
 *           cluster may share a tile's k ("split")
 *   WIDE    tensor cores, 256 channels x 256 tokens a CTA pair
 *   SLIM    as NARROW, up to 32 tokens
 * sgemm_fp4_tune_force(kernel) makes every later product in the process take
 * that kernel (AUTO: the rule again; a product the kernel cannot take follows
 * the rule); SGEMM_ERR_INVALID_ARG for an unknown one.  It is a process-wide
 * setting: do not change it while other threads call the library.
 * sgemm_fp4_last_kernel and sgemm_fp4_last_split_count return the kernel (AUTO:
 * none, of K == 0) and the CTAs that share a tile's k of the most recent
 * product enqueued in this process, racy across threads that call at the same
 * time. */
#define SGEMM_FP4_KERNEL_AUTO 0
#define SGEMM_FP4_KERNEL_FEW 1
#define SGEMM_FP4_KERNEL_NARROW 2
#define SGEMM_FP4_KERNEL_WIDE 3
#define SGEMM_FP4_KERNEL_SLIM 4
int sgemm_fp4_tune_force(int kernel);
int sgemm_fp4_last_kernel(void);
int sgemm_fp4_last_split_count(void);

#ifdef __cplusplus
}
#endif

#endif /* FP4_GEMM_GB300_H */
