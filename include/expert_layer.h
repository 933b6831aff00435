/*
 * expert_layer.h -- tokens sorted by expert and back, with weights applied,
 * and its gradient, on one GB300 (part of libsgemm_gb300.so; status codes as
 * in sgemm.h, row types as in int8_gemm.h).
 *
 * T tokens choose k experts each out of E: ids[t][j].  Choice s = t * k + j
 * gets position p(s) in an order sorted by expert, stable (an expert's
 * choices keep the order of s).  An id outside 0 .. E-1 is a dropped choice
 * (an expert over its capacity, or one held elsewhere): it sorts behind all
 * others and takes part in nothing.
 *
 *   sort           offsets[e] = first position of expert e (offsets[E] = the
 *                  number of kept choices), slots[p(s)] = s, positions[s] = p(s)
 *   dispatch       rows[p(t,j)] = x[t]                  (dropped: zeros)
 *   its gradient   dx[t] = sum_j drows[p(t,j)]          (kept j)
 *   combine        out[t] = sum_j w[t][j] rows[p(t,j)]  (kept j)
 *   its gradient   drows[p(t,j)] = w[t][j] dout[t]      (dropped: zeros)
 *                  dw[t][j] = sum_h rows[p(t,j)][h] dout[t][h]  (dropped: 0)
 *
 * Rows of dropped choices are never read: what they hold, NaN included, does
 * not reach a result.  A token whose choices are all dropped gets a row of
 * zeros.  Sums are fp32, in the order of j, rounded once to the row type; dw's
 * over h in an order fixed by the sizes and the alignment of all rows: repeated
 * calls give the same bits, calls on rows aligned differently may not.
 *
 * All matrices are row-major with leading dimensions in elements (>= H);
 * slots and positions have T * k entries, offsets E + 1; weights and dweights
 * are T x k fp32, contiguous.  Every pointer is a DEVICE pointer owned by the
 * caller; outputs may not overlap inputs or each other.  Any alignment of
 * rows to their type is accepted; rows on 16-byte boundaries are fastest.
 * 1 <= k <= 64, 1 <= E <= 1024, T * k < 2^31.  Calls enqueue on `stream` and
 * return; nothing is allocated or synchronised.
 *
 * Errors: SGEMM_ERR_INVALID_ARG (dimensions, type, NULL where data is read or
 * written, misaligned pointers) before anything is launched;
 * SGEMM_ERR_UNSUPPORTED without a compute capability 10.3 GPU;
 * SGEMM_ERR_LAUNCH if a launch fails.  T == 0: sort writes zero offsets, the
 * others do nothing.  H == 0: nothing but zero dweights and scales.
 */
#ifndef EXPERT_LAYER_GB300_H
#define EXPERT_LAYER_GB300_H

#include "int8_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* offsets, slots and positions of ids (T x k, contiguous, 32-bit). */
int sgemm_experts_sort(int T, int k, int E, const int *ids, int *offsets, int *slots,
                       int *positions, void *stream);

/* rows (T * k x H) from x (T x H). */
int sgemm_experts_dispatch(int type, int T, int k, int E, int H, const void *x, int ldx,
                           const int *positions, const int *offsets, void *rows, int ldr,
                           void *stream);

/* As sgemm_experts_dispatch, each token's row quantised on the way as
 * sgemm_i8_quantize_rows does it: codes q (T * k x H, 8-bit) and their scales
 * (T * k), in expert order, ready for sgemm_i8_experts. */
int sgemm_experts_dispatch_i8(int type, int T, int k, int E, int H, const void *x, int ldx,
                              const int *positions, const int *offsets, signed char *q, int ldq,
                              float *scale, void *stream);

/* dx (T x H) from drows (T * k x H): the gradient of dispatch. */
int sgemm_experts_dispatch_grad(int type, int T, int k, int E, int H, const void *drows, int ldr,
                                const int *positions, const int *offsets, void *dx, int ldx,
                                void *stream);

/* out (T x H) from rows (T * k x H); weights NULL means 1 everywhere. */
int sgemm_experts_combine(int type, int T, int k, int E, int H, const void *rows, int ldr,
                          const int *positions, const int *offsets, const float *weights,
                          void *out, int ldo, void *stream);

/* drows (T * k x H) and dweights (T x k; NULL: not wanted, rows is then not
 * read) from dout (T x H) and the rows and weights combine was given. */
int sgemm_experts_combine_grad(int type, int T, int k, int E, int H, const void *dout, int ldo,
                               const void *rows, int ldr, const int *positions,
                               const int *offsets, const float *weights, void *drows, int ldd,
                               float *dweights, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* EXPERT_LAYER_GB300_H */
