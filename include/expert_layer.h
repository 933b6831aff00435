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

/* A whole expert layer for a few tokens (a decoding step), in two kernels,
 * from the choices as they are: no sort, no rows in expert order.
 *
 *   h[t][j] = silu(x[t] G_e^T) * (x[t] U_e^T)        e = ids[t][j]
 *   out[t]  = sum_j weights[t][j] * (h[t][j] D_e^T)  (kept j)
 *
 * W1 holds G_e (rows 0 .. F-1) and U_e (rows F .. 2F-1) of every expert, 2F x H
 * at W1 + e * stride1 elements, W2 D_e, H x F at W2 + e * stride2; their type:
 *   SGEMM_EXPERTS_I8    8-bit integers with a scale per row, scale1 (E x 2F)
 *                       and scale2 (E x H), as sgemm_i8_experts takes them
 *   SGEMM_EXPERTS_SAME  the row type; scale1 and scale2 are not read
 * type is SGEMM_TYPE_BF16 or SGEMM_TYPE_FP16.  x, out: T x H, any alignment;
 * ids: T x k (an id outside 0 .. E-1 is a dropped choice; a token may choose
 * an expert twice); weights: T x k fp32, NULL means 1 everywhere.  Rows of W1
 * and W2 start on 16-byte boundaries (bases, leading dimensions and strides).
 * T <= 64, T * k <= 512, H and F <= 65536.
 * Products are exact where weights are 8-bit; sums are fp32; h is kept in two
 * values of the row type between the products, to twice its digits (fp16: to
 * 2^-36 at the least, and an h beyond 65504 is an infinity);
 * out is summed over the experts in fp32, in an order fixed by ids and the
 * sizes, and rounded once.  Only experts that a kept choice names are read.  A
 * token without kept choices gets zeros.  out may not overlap x.
 * workspace: 16-byte aligned, at least the size below (0 for sizes that the
 * layer refuses, too); a call does not read what it did not write there; calls
 * that may run at the same time need one each.
 * For more tokens there are the calls above: sort, dispatch_i8, sgemm_i8_experts
 * with W1, sgemm_i8_quantize_rows with SGEMM_ACT_SWIGLU, sgemm_i8_experts with W2,
 * combine.  They also round the activations to 8 bits, and with 8-bit weights are
 * the faster way from some eight tokens on (32 experts of 2048 x 1024, 4 a token,
 * us: 1 token 14 here, 25 there; 8 tokens 34, 35; 16 tokens 54, 43; 64 tokens 115,
 * 59). */
#define SGEMM_EXPERTS_I8 0
#define SGEMM_EXPERTS_SAME 1
size_t sgemm_experts_layer_workspace_size(int T, int k, int H, int F);
int sgemm_experts_layer(int type, int wtype, int T, int k, int E, int H, int F, const void *x,
                        int ldx, const int *ids, const float *weights, const void *W1, int ld1,
                        long long stride1, const float *scale1, const void *W2, int ld2,
                        long long stride2, const float *scale2, void *out, int ldo,
                        void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* EXPERT_LAYER_GB300_H */
