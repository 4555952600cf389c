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
 *   rotary       : rotary positions of queries and keys, and their gradient
 *   attention    : softmax attention over packed documents (causal, sliding
 *                  window, prefix, capped scores, distance bias, shared key-value
 *                  heads), and its gradient
 *   orthogonalize: Newton-Schulz products that bring a matrix's singular values
 *                  towards 1, for updates that are orthogonalised
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

/* ------------------------------------------------------------------ rotary -- */
#define LOWBIT_ROTARY_HALF 0         /* pairs (i, i + rot_dim / 2)              */
#define LOWBIT_ROTARY_INTERLEAVED 1  /* pairs (2 i, 2 i + 1)                    */

#define LOWBIT_ROTARY_PLAIN 0        /* f_i = base^(-2 i / rot_dim)             */
#define LOWBIT_ROTARY_LINEAR 1       /* f_i / factor                            */
#define LOWBIT_ROTARY_BASE 2         /* base * factor^(rot_dim / (rot_dim - 2)):
                                        the slowest pair is divided by factor,
                                        the fastest kept (rot_dim 2: kept)      */
#define LOWBIT_ROTARY_PARTS 3        /* f_i / factor for pairs of at most
                                        slow_turns over original_length
                                        positions, f_i for those of at least
                                        fast_turns, in between a mean whose weight
                                        is linear in the turns; rotated values are
                                        to be scaled by 0.1 ln(factor) + 1      */

/*
 * The rot_dim / 2 frequencies of a context that is scaled by `factor`, in
 * radians a position, and the scale that goes with them.  Host arithmetic only.
 *   freqs : host, rot_dim / 2 binary64 (written);  scale : host (written)
 * EINVAL: NULL pointer, rot_dim not an even number in 2 .. 65536, unknown scaling,
 * base or factor not above 0 or not finite, factor below 1 for LOWBIT_ROTARY_PARTS,
 * and there original_length < 1 or not 0 <= slow_turns < fast_turns.
 */
lowbit_status lowbit_rotary_frequencies(int32_t rot_dim, double base, int32_t scaling,
                                        double factor, int64_t original_length, double slow_turns,
                                        double fast_turns, double* freqs, float* scale);

/* Where the rows and heads of a matrix rows x heads x head_dim lie, in elements;
 * the elements of a head are dense. */
typedef struct {
    int64_t row, head;
} lowbit_strides;

typedef struct {
    int64_t rows;               /* tokens, up to 2^31 - 1                       */
    int64_t rows_per_sequence;  /* without `positions`: row r's is
                                   r mod rows_per_sequence (>= 1)               */
    lowbit_strides x, y;
    int32_t heads;              /* up to 65536                                  */
    int32_t head_dim;           /* up to 65536                                  */
    int32_t rot_dim;            /* even, 2 .. head_dim: the first elements of a
                                   head; the others are copied                  */
    int32_t layout;             /* LOWBIT_ROTARY_HALF or _INTERLEAVED           */
    int32_t type;               /* lowbit_dtype of x and y                      */
    float   scale;              /* of the rotated values                        */
} lowbit_rotary_params;

/*
 * Rotary positions: every pair (u, v) of a head of row r, of frequency f, gives
 *     scale * (u cos a - v sin a),  scale * (u sin a + v cos a),   a = position[r] f.
 *   x, y      : rows x heads x head_dim; y may be x, with equal strides, and then
 *               only the rotated part is read and written.  They need no alignment
 *               beyond the type's.
 *   freqs     : rot_dim / 2 binary64, device
 *   positions : rows int64, device, of any sign; NULL: counted
 * Angles are taken in binary64 and reduced before sine and cosine: exact to
 * 2^-22 of a turn up to positions of 2^30 and frequencies up to 1.
 * EINVAL: p == NULL, a size, type or option outside its range, a negative stride, strides
 * of y with which two of its elements share a place, y == x with unequal strides, NULL
 * or misaligned pointer with rows > 0.
 */
lowbit_status lowbit_rotary(const void* x, const double* freqs, const int64_t* positions,
                            const lowbit_rotary_params* p, void* y, hipStream_t stream);

/* Its gradient: dx from dy, the pairs turned back.  The strides x are dy's, y
 * are dx's; dx may be dy. */
lowbit_status lowbit_rotary_backward(const void* dy, const double* freqs,
                                     const int64_t* positions, const lowbit_rotary_params* p,
                                     void* dx, hipStream_t stream);

/* --------------------------------------------------------------- attention -- */
typedef struct {
    int64_t q_rows, k_rows;     /* of the buffers, up to 2^29                   */
    int64_t window;             /* 0: none                                      */
    int32_t sequences;          /* 0 .. 2^24                                    */
    int32_t q_heads, kv_heads;  /* up to 4096; kv_heads divides q_heads, and query
                                   head h reads key-value head
                                   h / (q_heads / kv_heads)                     */
    int32_t head_dim;           /* a multiple of 8, up to 128                   */
    int32_t type;               /* lowbit_dtype of everything but lse and slopes */
    int32_t causal;             /* 0 or 1                                       */
    float   scale;              /* of the products, finite                      */
    float   softcap;            /* 0: none; finite, >= 0                        */
    lowbit_strides q, k, v, out;
    lowbit_strides dout, dq, dk, dv;   /* the gradient's                        */
} lowbit_attention_params;

/* Bytes of workspace that the forward (backward = 0) or the backward call
 * (backward = 1) needs, or -1 for invalid params; 0 where it takes none. */
int64_t lowbit_attention_workspace(const lowbit_attention_params* p, int32_t backward);

/*
 * Attention.  Sequence s has the queries q_begin[s] .. q_begin[s + 1] - 1 and the
 * keys k_begin[s] .. k_begin[s + 1] - 1, Lq and Lk of them.  Its query i stands at
 * position i + Lk - Lq (the last query at the last key) and sees key j if
 *     j < prefix[s], or
 *     (not causal or j <= position) and (no window or |position - j| < window).
 * Of those it sees
 *     y_j = softcap * tanh(scale q.k_j / softcap) - slopes[head] |position - j|
 *     lse = log sum_j exp(y_j),    out = sum_j exp(y_j - lse) v_j;
 * a query that sees none has out = 0 and lse = -infinity.
 *   q, out : q_rows x q_heads x head_dim;  k, v : k_rows x kv_heads x head_dim
 *   lse    : q_heads x q_rows binary32, dense
 *   q_begin, k_begin : sequences + 1 int32, device, not decreasing, from 0 up to at
 *            most q_rows (k_rows); values beyond are cut to that.  Rows before the
 *            first and behind the last sequence are not written, and nothing depends on
 *            what they hold.  Both
 *            NULL: sequences of q_rows / sequences queries and k_rows / sequences keys
 *            each (they have to divide); k_begin NULL: the same as q_begin (then
 *            k_rows == q_rows); q_begin NULL alone: queries in equal sequences.
 *            Offsets that decrease give unspecified results within the buffers.
 *   prefix : sequences int32, device, or NULL: 0 for all
 *   slopes : q_heads binary32, device, or NULL: 0 for all
 * Rows' strides are multiples of 8 elements from head_dim up to 2^22, heads' strides
 * multiples of 8; two elements of an output share no place.
 * Scores, statistics and sums are binary32 (of LOWBIT_BF16, scores beyond half their softcap
 * are off by up to 2^-20, relative).  For LOWBIT_BF16 the weights exp(y - m) (m near the largest
 * so far) enter the product with v rounded to bfloat16, off by up to 2^-8 each, relative.  NaN and infinities of a key or value that a query does not
 * see reach it only within its own sequence.
 * EINVAL: p == NULL, a size, type, option or stride outside its range, NULL or
 * misaligned pointer with rows and sequences > 0, workspace too small.  EUNSUPPORTED: head_dim above 128.
 */
lowbit_status lowbit_attention(const void* q, const void* k, const void* v,
                               const int32_t* q_begin, const int32_t* k_begin,
                               const int32_t* prefix, const float* slopes,
                               const lowbit_attention_params* p, void* out, float* lse,
                               void* workspace, int64_t workspace_bytes, hipStream_t stream);

/*
 * Its gradient, from the gradient of out and the forward call's out and lse:
 *     D = sum_d dout out,   g_j = exp(y_j - lse) (dout.v_j - D) (1 - tanh^2),
 *     dq = scale sum_j g_j k_j,  dk_j = scale sum_i g_ij q_i,  dv_j = sum_i exp(y_ij - lse_i) dout_i,
 * the last two over every query head that reads j's head.  lse and the slopes have no
 * gradient here.  A key that no query sees has dk = dv = 0; rows outside all sequences are left as they
 * were.  For LOWBIT_BF16 the weights and g enter their products rounded to
 * bfloat16, as in the forward call.
 * Equal calls give equal bits.  Where sums are cut into parts follows from the buffers'
 * sizes, not from the offsets: the same rows within larger buffers may differ by the rounding of
 * binary32 additions in another order (so also of the forward call).
 */
lowbit_status lowbit_attention_backward(const void* dout, const void* q, const void* k,
                                        const void* v, const void* out, const float* lse,
                                        const int32_t* q_begin, const int32_t* k_begin,
                                        const int32_t* prefix, const float* slopes,
                                        const lowbit_attention_params* p, void* dq, void* dk,
                                        void* dv, void* workspace, int64_t workspace_bytes,
                                        hipStream_t stream);

/* ----------------------------------------------------------- orthogonalize -- */
typedef struct {
    int64_t batch;              /* matrices, up to 2^20                         */
    int64_t rows, cols;         /* of each, 1 .. 65536; up to 2^40 elements in all */
    int32_t type;               /* lowbit_dtype of g                            */
    int32_t steps;              /* 0 .. 64                                      */
    float   a, b, c;            /* coefficients, finite                         */
    float   eps;                /* >= 0                                         */
    float   scale;              /* of the result, finite                        */
} lowbit_orthogonalize_params;

/* Bytes of workspace that lowbit_orthogonalize needs, or -1 for invalid params. */
int64_t lowbit_orthogonalize_workspace(const lowbit_orthogonalize_params* p);

/*
 * Newton-Schulz.  Of each matrix
 *     X = g / (sqrt(sum g^2) + eps);   `steps` times  A = X X^T, X = a X + (b A + c A A) X;
 *     out = scale X                    (for rows > cols: of g's transpose, turned back)
 * With a = 3.4445, b = -4.7750, c = 2.0315 (the coefficients that K. Jordan published with the
 * Muon optimizer, 2024) five steps bring all but the smallest singular values to between 0.7 and 1.2.
 *   g   : batch x rows x cols, of p->type
 *   out : batch x rows x cols bfloat16 (written); may be g where that is bfloat16
 * X is held in binary32 throughout.  The products' operands (X, A, b A + c A A) are rounded
 * to binary16, scaled by powers of two against its range, off by up to 2^-11 each,
 * relative, and summed in binary32: three bits more than
 * bfloat16 operands, whose errors the iteration raises to several hundredths.  They hold singular
 * values up to 4; coefficients that let X grow beyond give infinities or NaN.  A matrix of zeros gives
 * zeros if eps > 0, one with an infinity or NaN gives NaN (from the first step on).
 * EINVAL: p == NULL, a size, type or option outside its range, NULL or misaligned
 * pointer with batch > 0, workspace too small.
 */
lowbit_status lowbit_orthogonalize(const void* g, const lowbit_orthogonalize_params* p, void* out,
                                   void* workspace, int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LOWBIT_TRAIN_H */
