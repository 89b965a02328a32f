/*
 * onetrans_input.h - C ABI of the OneTrans input layer on B200 (sm_100a):
 * embedding tables and the routed event tokenizer, each with its gradient.
 * They lead from item ids to the S-tokens that onetrans_stage1_encode,
 * onetrans_forward and onetrans_forward_backward take, and from the input
 * gradient that onetrans_forward_backward writes back to the tables:
 *
 *   ids -> onetrans_embedding_lookup -> events -> onetrans_route_events,
 *   onetrans_tokenize_routed -> S-tokens -> the block stack -> dx0
 *   -> onetrans_tokenize_routed_backward -> event gradients
 *   -> onetrans_embedding_backward(_sparse) -> table gradients
 *
 * The conventions of onetrans.h hold: device pointers owned by the caller and
 * 16-byte aligned (workspaces and plans 256-byte), the model's mode as element
 * type unless said otherwise, nothing allocated, calls asynchronous on
 * `stream`, argument errors found on the host before any launch, a call with
 * no work returns ONETRANS_OK and launches nothing.  Every call may be
 * captured into a CUDA graph.  Two calls that may run at the same time need
 * workspaces (and plans, unless both only read one) of their own; that
 * includes two graphs that are replayed at the same time.  Sums are float32
 * and added in a fixed order: equal inputs give equal bits.
 */
#ifndef ONETRANS_INPUT_H
#define ONETRANS_INPUT_H

#include "onetrans.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Which buffer onetrans_input_workspace_size() sizes.  A buffer of that size
 * also serves calls with fewer ids or events (of the same or a smaller L). */
typedef enum {
  ONETRANS_OP_EMBEDDING_BACKWARD = 0, /* n = R ids,    L = width */
  ONETRANS_OP_ROUTE = 1,              /* the plan: n = R events, L = k */
  ONETRANS_OP_ROUTED = 2,             /* n = R events, L = k */
  ONETRANS_OP_ROUTED_BACKWARD = 3     /* n = R events, L = k */
} onetrans_input_op;

ONETRANS_API onetrans_status onetrans_input_workspace_size(const onetrans_model* m, int32_t op, int64_t n,
                                                           int32_t L, size_t* bytes);

/* ------------------------------------------------------- embedding tables --
 * The tables are arguments, not part of the model, and stay the caller's.
 * ids: int32 (ids_bits 32) or int64 (ids_bits 64).  Id -1 is padding; any
 * other id outside 0 .. n_rows-1 counts as padding too and sets the device
 * status word (code 3).  n_rows <= 2^31 - 1, width <= 65536. */

/* out[r] = scale * table[ids[r]] (a zero row for padding), R rows.
 *   table [n_rows, width] of element type table_mode (ONETRANS_BF16 or
 *   ONETRANS_FP32); out: rows of the mode's type, out_ld >= width elements
 *   apart, 4-byte aligned (so that the fields of one feature row can be
 *   looked up side by side); what lies between two rows is left as it was.  The product is
 *   taken in float32 and rounded once. */
ONETRANS_API onetrans_status onetrans_embedding_lookup(const onetrans_model* m, const void* table,
                                                       int32_t table_mode, int64_t n_rows, int32_t width,
                                                       const void* ids, int32_t ids_bits, int64_t R, float scale,
                                                       void* out, int64_t out_ld, void* stream);

/* The gradient of a lookup, dense: dtable[v] = scale * (sum of dout[r] over
 * the r with ids[r] = v), float32, every row of dtable [n_rows, width]
 * written (zeros where no id names it).
 *   dout: rows of element type dout_mode, dout_ld >= width elements apart,
 *     4-byte aligned (the columns of one field of a wider gradient).
 * R = 0 still writes the zeros.  R <= 2^26.  Workspace:
 * ONETRANS_OP_EMBEDDING_BACKWARD. */
ONETRANS_API onetrans_status onetrans_embedding_backward(const onetrans_model* m, const void* dout,
                                                         int32_t dout_mode, int64_t dout_ld, const void* ids,
                                                         int32_t ids_bits, int64_t R, int64_t n_rows,
                                                         int32_t width, float scale, float* dtable, void* ws,
                                                         size_t ws_bytes, void* stream);

/* The same gradient as the touched rows only: uniq[i] (the ids' type)
 * ascending, rows[i] [width] float32 the sum of row uniq[i], i < *n_uniq.
 * uniq and rows have room for min(R, n_rows) rows; rows at and behind *n_uniq
 * are left as they were.  n_uniq: int32 on the device (16-byte aligned like
 * every buffer).  R = 0 writes *n_uniq = 0. */
ONETRANS_API onetrans_status onetrans_embedding_backward_sparse(
    const onetrans_model* m, const void* dout, int32_t dout_mode, int64_t dout_ld, const void* ids,
    int32_t ids_bits, int64_t R, int64_t n_rows, int32_t width, float scale, void* uniq, float* rows,
    int32_t* n_uniq, void* ws, size_t ws_bytes, void* stream);

/* -------------------------------------------------- routed event tokenizer --
 * Event r stands for up to k behaviours: its token is the weighted sum of its
 * behaviours' tokens,
 *   token[r] = sum_j weights[r][j] * (W2_t GELU(W1_t e_r + b1_t) + b2_t + emb_t),
 * t = types[r][j], with the per-behavior MLPs and type identifiers of the
 * model (Wb1, bb1, Wb2, bb2, type_emb; GELU in its tanh form).  With k = 1
 * and no weights this is onetrans_tokenize_events' function; that call
 * computes every behaviour's MLP for every event, these sort the events by
 * behaviour and compute each event's own.  UNSUPPORTED when the model has no
 * behavior MLPs or no type_emb.  1 <= k <= 8, R * k <= 2^26. */

/* Sorts the choices by behaviour into `plan` (a caller's buffer of
 * ONETRANS_OP_ROUTE bytes, 256-byte aligned), which the two calls below read
 * for the same R and k.  types [R, k] int32 (device): 0 .. n_behaviors-1, or
 * -1 for a choice that is none (it takes no part; a row of them gives a zero
 * token).  Any other id counts as -1 and sets the device status word (code
 * 3).  A behaviour may occur twice in a row. */
ONETRANS_API onetrans_status onetrans_route_events(const onetrans_model* m, const int32_t* types, int64_t R,
                                                   int32_t k, void* plan, size_t plan_bytes, void* stream);

/* tokens of R events.
 *   events [R, event_dim] (mode's type); weights [R, k] float32 or NULL (1);
 *   tokens (mode's type): row r at (r / rows_per_sample) * sample_ld +
 *     (r % rows_per_sample) * d elements, so that the S rows of x0
 *     [B, L_S + L_NS, d] are written in place (rows_per_sample = L_S,
 *     sample_ld = (L_S + L_NS) * d); rows_per_sample >= R: rows one after
 *     another, sample_ld is not looked at.  Elements outside those rows are
 *     left as they were.
 * A plan that onetrans_route_events did not make for this model's behaviours,
 * R and k sets the device status word (code 3) and nothing is written.
 * Sums are float32, the token is rounded once.  BF16 mode with d_model a
 * multiple of 64 up to 384, event_dim a multiple of 16 up to 128 and sample_ld
 * a multiple of 8 runs on tensor cores: the hidden row z is rounded to bf16 as
 * the operand of the second product, and its GELU is off by up to 2^-12 |u|
 * more.  Other shapes keep z in float32. */
ONETRANS_API onetrans_status onetrans_tokenize_routed(const onetrans_model* m, const void* events,
                                                      const float* weights, int64_t R, int32_t k, const void* plan,
                                                      size_t plan_bytes, void* tokens, int64_t rows_per_sample,
                                                      int64_t sample_ld, void* ws, size_t ws_bytes, void* stream);

/* Gradients of the behaviour weights (float32, each with its weight's shape;
 * host arrays of n_behaviors device pointers, type_emb [n_behaviors, d]).
 * Written, not accumulated. */
typedef struct {
  float* const* Wb1;
  float* const* bb1;
  float* const* Wb2;
  float* const* bb2;
  float* type_emb;
} onetrans_event_grads;

/* The gradient of onetrans_tokenize_routed for the upstream gradient dtokens
 * (laid out like tokens; element type dtokens_mode: ONETRANS_FP32, as
 * onetrans_forward_backward writes dx0, or in BF16 mode ONETRANS_BF16):
 *   devents [R, event_dim] (mode's type) or NULL;
 *   dweights [R, k] float32 or NULL (0 where a choice is none);
 *   grads: every weight gradient (zeros for a behaviour without events).
 * BF16 mode: float32 dtokens are rounded to bf16 as matrix operands.  On tensor
 * cores (the shapes above) z and the pre-activation gradient enter the weight
 * gradients' products as two bf16 terms (16 bits of significand; an infinity in
 * dtokens or events, which meets two terms of either sign, can make NaN where
 * the product is infinite), and the event gradient's product as one, rounded
 * once more as devents are stored.  Other shapes keep both in float32.  R = 0
 * writes the zeros of grads.  The plan is checked as above. */
ONETRANS_API onetrans_status onetrans_tokenize_routed_backward(
    const onetrans_model* m, const void* events, const float* weights, int64_t R, int32_t k, const void* plan,
    size_t plan_bytes, const void* dtokens, int32_t dtokens_mode, int64_t rows_per_sample, int64_t sample_ld,
    void* devents, float* dweights, const onetrans_event_grads* grads, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* ONETRANS_INPUT_H */
