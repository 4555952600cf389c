/*
 * lowbit_train.h -- C ABI of liblowbit's training-step operators on AMD
 * Instinct MI355X (gfx950): the steps between which a data-parallel rank's
 * gradients come into being before the codec of lowbit.h compresses them.
 *
 *   dropout      : y = residual + D(x), and its gradient; the mask is drawn
 *                  from the library's counter hash and never stored
 *   block join   : between two blocks of a residual network,
 *                      x_out = a x + gate * D(norm(f)),  z = norm(x_out),
 *                  and its gradient
 *   linear xent  : softmax cross entropy of x w^T over a large vocabulary
 *                  without keeping the logits, and its gradient
 *
 * The mask.  Element i of a buffer (for a matrix of `cols` columns, row r's
 * column c counts as i = r * (cols + cols mod 2) + c) belongs to pair i / 2,
 * whose word is h = fmix32(lo32(i / 2) ^ fmix32(hi32(i / 2) ^ K(seed))), fmix32
 * and K as in lowbit.h; its draw is the low half of h for even i, the high half
 * for odd i.  With t = p * 65536 rounded to nearest (ties to even), D keeps the
 * elements whose draw is at least t, multiplied by 65536 / (65536 - t) (by 0 if
 * t = 65536), and gives +0 elsewhere, whatever stood there.
 * Masks of two seeds are not independent of each other: below 2^33 elements pair
 * q's word is fmix32(q ^ c) with c = fmix32(K(seed)), so that another seed's mask
 * has the word of pair q at pair q ^ c ^ c'.  Two buffers of 2^25 pairs hold the same
 * words in another order for one pair of seeds in 128 (of 2^m pairs: one in
 * 2^(32 - m)), smaller or larger parts of them for others.
 *
 * Conventions of lowbit.h hold: device pointers, element buffers (x, y, f,
 * w, gradients, parameters, gate, lse, ...) aligned to 16 bytes, targets to 8;
 * asynchronous launches on `stream`; argument errors returned before anything
 * is launched; outputs must not overlap inputs or each other unless stated.
 * Matrices are dense and row-major.  The library allocates nothing: calls with
 * scratch take `workspace`, aligned to 16 bytes, of at least the bytes that the
 * matching *_workspace function gives.  It holds nothing between calls, and two
 * calls that may run at the same time need one each.  Arithmetic, sums and
 * statistics are binary32 and each output is rounded once; one value in between is
 * held in fewer bits, d of linear xent's gradient (below).  Sums run in a fixed
 * order, so that equal calls give equal bits.  Every call can be captured into a
 * HIP graph.
 */
#ifndef LOWBIT_TRAIN_H
#define LOWBIT_TRAIN_H

#include "lowbit.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Dropout:  y = residual + D(x)   (residual NULL: y = D(x)).
 *   x, residual, y : n elements of type t; y may be x or residual itself
 *   p              : in [0, 1]
 *   index_offset   : index of element 0 in the mask, a multiple of 8, so that a
 *                    buffer split at such places draws the same mask
 * EINVAL: n < 0 or above 2^48, p not in [0, 1], bad index_offset, unknown type,
 * NULL or misaligned pointer with n > 0.
 */
lowbit_status lowbit_dropout(const void* x, const void* residual, lowbit_dtype t, int64_t n,
                             double p, uint64_t seed, uint64_t index_offset, void* y,
                             hipStream_t stream);

/* Its gradient: dx = D(dy) with the forward call's p, seed and index_offset
 * (the residual's gradient is dy itself). */
lowbit_status lowbit_dropout_backward(const void* dy, lowbit_dtype t, int64_t n, double p,
                                      uint64_t seed, uint64_t index_offset, void* dx,
                                      hipStream_t stream);

#define LOWBIT_NORM_RMS 0     /* v / sqrt(mean(v^2) + eps)                        */
#define LOWBIT_NORM_LAYER 1   /* (v - mean(v)) / sqrt(var(v) + eps), var over cols */

typedef struct {
    int64_t rows;
    int64_t cols;             /* 1 .. 16384                                    */
    int64_t rows_per_gate;    /* consecutive rows that share a row of the gate;
                                 used only where a gate is given; any number
                                 from `rows` on: one row for all               */
    int32_t norm;             /* LOWBIT_NORM_*                                 */
    int32_t block_type;       /* lowbit_dtype of f, z and their gradients      */
    int32_t stream_type;      /* of x, x_out and their gradients: block_type
                                 or LOWBIT_F32                                 */
    int32_t param_type;       /* of weights, biases and gate: block_type or
                                 LOWBIT_F32                                    */
    float   eps;              /* >= 0                                          */
    float   residual_scale;   /* a                                             */
    double  p;                /* dropout, in [0, 1]; 0: none                   */
    uint64_t seed;
} lowbit_join_params;

/*
 * Block join.  For every row
 *     u     = norm(f) * post_weight + post_bias
 *     x_out = a x + gate[row / rows_per_gate] * D(u)
 *     z     = norm(x_out) * pre_weight + pre_bias
 * the second norm taken before x_out is rounded.  post_weight, post_bias,
 * gate, pre_weight, pre_bias may be NULL (1, 0, 1, 1, 0).
 *   f, x       : rows x cols;  weights and biases: cols
 *   gate       : ceil(rows / rows_per_gate) x cols
 *   x_out, z   : rows x cols (written); x_out may be x, z may be f
 *   stats      : rows x 4 binary32 (written): mean and 1/sqrt(var + eps) of f's
 *                row, then of x_out's (means 0 for LOWBIT_NORM_RMS)
 * EINVAL: p == NULL, a size, type or option outside its range, NULL or
 * misaligned pointer with rows > 0.  EUNSUPPORTED: more than 16384 columns.
 */
lowbit_status lowbit_block_join(const void* f, const void* x, const void* post_weight,
                                const void* post_bias, const void* gate, const void* pre_weight,
                                const void* pre_bias, const lowbit_join_params* p, void* x_out,
                                void* z, float* stats, hipStream_t stream);

/* Bytes of workspace that lowbit_block_join_backward needs, or -1 for invalid
 * params. */
int64_t lowbit_block_join_backward_workspace(const lowbit_join_params* p);

/*
 * Gradient of the block join, from the gradients of x_out and z, the forward
 * call's f, x_out and stats and its parameters (p and seed redraw the mask).  The
 * second norm's gradient is taken at x_out as it was written, rounded to
 * stream_type, with the statistics of the row before it was rounded.
 *   df, dx : rows x cols (written); df may be dz, dx may be dx_out
 *   dpost_weight, dpost_bias, dpre_weight, dpre_bias : cols binary32 each;
 *   dgate  : ceil(rows / rows_per_gate) x cols binary32 (only with a gate).
 * Any of these five may be NULL and is then not computed; those given are
 * written whatever parameters are NULL (the gradient at 1 or 0), with zeros for
 * rows == 0.
 */
lowbit_status lowbit_block_join_backward(const void* dx_out, const void* dz, const void* f,
                                         const void* x_out, const float* stats,
                                         const void* post_weight, const void* post_bias,
                                         const void* gate, const void* pre_weight,
                                         const lowbit_join_params* p, void* df, void* dx,
                                         float* dpost_weight, float* dpost_bias, float* dgate,
                                         float* dpre_weight, float* dpre_bias, void* workspace,
                                         int64_t workspace_bytes, hipStream_t stream);

typedef struct {
    int64_t rows;             /* tokens, up to 2^30                            */
    int64_t vocab;            /* 1 .. 2^31 - 1                                 */
    int64_t hidden;           /* 1 .. 2^20                                     */
    int64_t ignore_index;     /* rows with this target are left out            */
    int32_t type;             /* lowbit_dtype of x, w and their gradients      */
} lowbit_xent_params;

/* Bytes of workspace that the forward (backward = 0) or the backward call
 * (backward = 1) needs, or -1 for invalid params. */
int64_t lowbit_linear_xent_workspace(const lowbit_xent_params* p, int32_t backward);

/*
 * Softmax cross entropy of the logits l = x w^T:
 *     lse[r] = log sum_v exp(l[r, v]),   loss[r] = lse[r] - l[r, targets[r]]
 * and 0 for both in rows that are left out.  A target outside [0, vocab) that
 * is not ignore_index gives NaN for both, and so does a logit of +infinity or NaN;
 * logits of -infinity add nothing.
 *   x : rows x hidden;  w : vocab x hidden;  targets : rows int64
 *   loss, lse : rows binary32 (written)
 * Logits are binary32 sums of exact products.
 * EINVAL: p == NULL, a size or type outside its range, NULL or misaligned
 * pointer with rows > 0, workspace too small.
 */
lowbit_status lowbit_linear_xent(const void* x, const void* w, const int64_t* targets,
                                 const lowbit_xent_params* p, float* loss, float* lse,
                                 void* workspace, int64_t workspace_bytes, hipStream_t stream);

/*
 * Its gradient, from the forward call's lse and the gradients of loss and lse
 * (dlse NULL: zero; one is there for losses that use lse, as mean(lse^2)).  With
 *     d[r, v] = exp(l[r, v] - lse[r]) (dloss[r] + dlse[r]) - dloss[r] [v = targets[r]]
 * it gives  dx = d w  and  dw = d^T x; d is formed in pieces of the vocabulary in
 * the workspace.  For LOWBIT_BF16 d is kept there in bfloat16, scaled so that
 * the largest |dloss| counts as 1: each of its elements is off by up to 2^-8 more,
 * relative, and so is an element of dx or dw that one of them makes up.  Rows that are left out give dx = 0 and add
 * nothing to dw; a target out of range gives NaN.
 *   dx : rows x hidden, dw : vocab x hidden, of type p->type; either may be NULL
 *        and is then not computed.  rows == 0 still writes dw (zeros).
 */
lowbit_status lowbit_linear_xent_backward(const void* x, const void* w, const int64_t* targets,
                                          const float* lse, const float* dloss, const float* dlse,
                                          const lowbit_xent_params* p, void* dx, void* dw,
                                          void* workspace, int64_t workspace_bytes,
                                          hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LOWBIT_TRAIN_H */
