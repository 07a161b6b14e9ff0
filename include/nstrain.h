/*
 * nstrain.h -- operators of a model trained on the library's packed rows.
 *
 * A packed batch's position ids, document ids and loss mask decide what a
 * model may mix, count and learn.  The operators declared here take them as
 * ns_pack_step writes them:
 *  - pos == 0 starts a new sequence within a row (ns_pack_out.pos);
 *  - doc < 0 is padding (ns_pack_out.doc);
 *  - mask == 0 is a position that is not learned (ns_pack_out.mask; for the
 *    loss of a position's next token, the mask of the next position).
 *
 *  - ns_scan_forward / ns_scan_backward: a gated linear recurrence over time
 *    that starts again at every sequence and passes over padding;
 *  - ns_distill: the divergence from a teacher's top logits on the learned
 *    positions, and its gradient in the same pass;
 *  - ns_route_forward / ns_route_backward: a router's choice of experts, the
 *    experts' counts and the balance loss over the real positions, and the
 *    logits' gradient.
 *
 * Conventions:
 *  - Every argument is checked on the host before anything is enqueued; a
 *    failing check returns NS_ERR_INVALID_ARG and changes nothing.  A launch
 *    that fails returns NS_ERR_CUDA.
 *  - All pointers are device memory of the current device, aligned for their
 *    element type; an optional one may be NULL.  Nothing is allocated, and
 *    the calls only enqueue kernels on cuda_stream (NULL: the legacy default
 *    stream).
 *  - Element types: NS_F32, NS_BF16, NS_F16.  States, sums, softmax
 *    statistics and losses are 32-bit floats; an output of 16 bits is rounded
 *    once, from 32 bits.
 *  - Every sum is taken in a fixed order: the same arguments give the same
 *    bits, on every call and every stream.  What a row (of a scan, of logits)
 *    gets does not depend on the other rows of the call; the order of a sum
 *    over rows (dbias, the balance loss) depends on the sizes and on the
 *    alignment of the arrays.
 *  - Values at padded or unlearned positions are never used, whatever they
 *    are (NaN and infinities among them); the outputs there are 0 (-1 for
 *    expert ids).
 */
#ifndef NSTRAIN_H
#define NSTRAIN_H

#include <stdint.h>

#include "nspack.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- element types -------------------------------------------------------- */
#define NS_F32 0
#define NS_BF16 1
#define NS_F16 2

/* ---- limits ---------------------------------------------------------------- */
#define NS_SCAN_TILE 32u         /* time steps between two saved states */
#define NS_SCAN_MAX_T (1u << 30) /* time steps of a row */
#define NS_DISTILL_MAX_TOP 1024u /* teacher logits a row */
#define NS_DISTILL_MAX_ROW (8u * 200u * 1024u) /* bytes of a row of logits */
#define NS_DISTILL_WIDE_ROW (8u * 176u * 1024u) /* beyond these, at most ... */
#define NS_DISTILL_WIDE_TOP 256u               /* ... so many teacher logits */
#define NS_ROUTE_MAX_EXPERTS 1024u
#define NS_ROUTE_MAX_K 32u       /* experts a token */

/* ---- gated linear recurrence ------------------------------------------------
 *   a_t = sigmoid(f_t + bias)                         per row, time and channel
 *   p_t = 0 where pos_t == 0, else h_{t-1};  h_{-1} = h0 (0 if NULL)
 *   h_t = a_t p_t + (1 - a_t) z_t,           y_t = h_t
 * and at padding (doc_t < 0) h_t = h_{t-1}, y_t = 0.  h_last is the state
 * after the last step: h0 where a row has no real position.  A row whose
 * first position id is not 0 goes on from h0.
 *
 * z and f are [B][T][D] with the channels contiguous and strides (in
 * elements) over rows and time; the halves of one projection are given as
 * they lie.  y, dz and df are contiguous [B][T][D]; bias is [D], h0 and
 * h_last [B][D], pos and doc contiguous [B][T] (either may be NULL: no
 * sequence starts, no padding).  h_last may be h0; no other output may overlap
 * an input.
 *
 * states ([B][ceil(T / NS_SCAN_TILE)][D] floats, NULL if no gradient is
 * wanted) receives the state before every tile of NS_SCAN_TILE steps; the
 * backward pass computes the states inside a tile again from it. */
typedef struct {
  const void *z;
  const void *f;
  int64_t z_row, z_time; /* strides of z, in elements */
  int64_t f_row, f_time; /* strides of f */
  const float *bias;     /* [D] or NULL */
  const int32_t *pos;    /* [B][T] or NULL */
  const int32_t *doc;    /* [B][T] or NULL */
  uint32_t B, T, D;      /* T <= NS_SCAN_MAX_T; any may be 0 */
  int32_t dtype;         /* of z, f, y and their gradients */
} ns_scan_inputs;

/* Errors: INVALID_ARG (a needed pointer NULL or misaligned, an unknown type,
 * a negative stride, sizes out of range), CUDA. */
int ns_scan_forward(const ns_scan_inputs *in, const float *h0, void *y, float *h_last,
                    float *states, void *cuda_stream);

/* Bytes of the workspace of ns_scan_backward for these sizes (0: none). */
uint64_t ns_scan_workspace(uint32_t B, uint32_t T, uint32_t D);

/* The gradients, from dy ([B][T][D], strides in elements) and dh_last
 * ([B][D] or NULL) and the states that the forward pass saved:
 *   d_t = dy_t + u_t, u_{t-1} = a_t d_t (0 where pos_t == 0), u_{T-1} = dh_last
 *   dz_t = (1 - a_t) d_t,  df_t = a_t (1 - a_t) d_t (p_t - z_t)
 *   dbias = the sum of df over rows and time, dh0 = u_{-1}
 * dbias ([D]) and dh0 ([B][D]) may be NULL.  No output may overlap an
 * input.  workspace: ns_scan_workspace bytes, 4-byte aligned; it may be NULL
 * where dbias is.  Errors: as ns_scan_forward. */
int ns_scan_backward(const ns_scan_inputs *in, const float *states, const void *dy,
                     int64_t dy_row, int64_t dy_time, const float *dh_last, void *dz, void *df,
                     float *dbias, float *dh0, void *workspace, void *cuda_stream);

/* ---- distillation from a teacher's top logits ---------------------------------
 * Row n has the student's logits s (V of them) and the teacher's K top logits
 * t with their token ids.  An entry whose id is outside [0, V) is absent.
 *   p_k = softmax over the row's entries of t_k / temperature
 *         or, with teacher_lse, exp(t_k / temperature - teacher_lse[n]): the
 *         teacher's own probabilities, whose sum m is below 1
 *   q   = softmax over V of s / temperature
 *   loss[n] = temperature^2 sum_k p_k (log p_k - log q_{id_k})
 *   dlogits[n][v] = weight[n] temperature (m q_v - sum of p_k with id_k = v)
 * (weight[n]: the gradient of what is minimised with respect to loss[n]; NULL
 * is 1.)  An entry of p_k = 0 adds nothing; one with p_k > 0 whose student
 * logit is -inf makes the loss infinite.  Where mask[n] is 0, or no entry is
 * left, the loss and the gradient are 0; an unlearned row is not read.
 *
 * Rows of logits and dlogits are strided (in elements); dlogits may be logits
 * itself (the gradient takes the logits' place), and NULL asks for the loss
 * alone.  top_logits, top_ids are contiguous [N][K]; ids may repeat. */
typedef struct {
  const void *logits;
  int64_t logits_row;      /* elements between rows, >= V */
  const void *top_logits;  /* [N][K], type top_dtype */
  const void *top_ids;     /* [N][K], int32, or int64 where ids_64 != 0 */
  const float *teacher_lse; /* [N] or NULL */
  const uint8_t *mask;     /* [N] or NULL: every row is learned */
  const float *weight;     /* [N] or NULL */
  uint32_t N, V, K;        /* N < 2^28, V * element size <= NS_DISTILL_MAX_ROW,
                              K <= NS_DISTILL_MAX_TOP (see NS_DISTILL_WIDE_ROW) */
  int32_t dtype, top_dtype;
  int32_t ids_64;
  float temperature;       /* > 0, finite */
} ns_distill_inputs;

/* Errors: INVALID_ARG (a needed pointer NULL or misaligned, an unknown type,
 * strides below V, sizes or temperature out of range), CUDA. */
int ns_distill(const ns_distill_inputs *in, float *loss, void *dlogits, int64_t dlogits_row,
               void *cuda_stream);

/* ---- router: experts, counts, balance loss -------------------------------------
 * Token n has E logits; p is their softmax.  Its k experts are the k largest
 * logits (of equal ones the lowest index first), in that order; an expert
 * whose logit is -inf is never chosen (id -1, weight 0), and a token whose
 * logits are all -inf, or with doc[n] < 0, chooses none and counts for nothing.
 * A NaN logit is never chosen and makes its token's weights, and the loss, NaN.
 *   weights = p at the chosen experts, with `normalize` divided by their sum
 *   counts[e] = tokens that chose e,  tokens[0] = M, the tokens that count
 *   loss = E / (k M^2) sum_e counts[e] sum_n p[n][e]   (0 if M = 0; 1 when
 *          experts are chosen evenly and their mean probabilities are equal)
 * logits rows are strided (in elements); ids and weights are contiguous
 * [N][k], counts [E]. */
typedef struct {
  const void *logits;
  int64_t logits_row;  /* elements between rows, >= E */
  const int32_t *doc;  /* [N] or NULL */
  uint32_t N, E, k;    /* N * k < 2^31; 1 <= k <= E */
  int32_t dtype;
  int32_t normalize;
} ns_route_inputs;

/* Bytes of the workspace of ns_route_forward for these sizes (0: none, or sizes that it
 * refuses). */
uint64_t ns_route_workspace(uint32_t N, uint32_t E);

/* workspace: ns_route_workspace bytes, 4-byte aligned, or NULL for none.  Errors: INVALID_ARG (a
 * needed pointer NULL or misaligned, an unknown type, sizes out of range), CUDA. */
int ns_route_forward(const ns_route_inputs *in, int32_t *ids, float *weights, int32_t *counts,
                     int32_t *tokens, float *loss, void *workspace, void *cuda_stream);

/* dlogits ([N][E], contiguous, the logits' type) from d_weights ([N][k] or
 * NULL) and d_loss (one float on the device, or NULL), with the forward
 * pass's outputs.  The counts do not depend on the logits (their gradient is
 * 0 wherever they have one).  Errors: as ns_route_forward. */
int ns_route_backward(const ns_route_inputs *in, const int32_t *ids, const float *weights,
                      const int32_t *counts, const int32_t *tokens, const float *d_weights,
                      const float *d_loss, void *dlogits, void *cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* NSTRAIN_H */
