/*
 * policy.h -- C ABI of the operators of a policy with memory in librollout.so
 * (gfx950), from the previous action to the next action's logits:
 *   embed_*   scaled embedding lookup, its gradient summed by sorted index
 *   recur_*   gated linear recurrence over a rollout, its gradient, its step
 *   logits_*  penalties, bias and mask on logits, and their gradient
 * Same conventions as rollout.h: DEVICE buffers owned by the caller,
 * asynchronous on the given stream (NULL = the default stream), ROLLOUT_OK or
 * a negative ROLLOUT_E* code with the message in rollout_last_error(), checks
 * on the host before anything is enqueued, no CPU fallback.  No call
 * allocates or keeps anything between calls: what a call needs besides its
 * buffers is the caller's workspace, whose size the *_workspace functions
 * give.  A workspace may be reused as soon as the call's work is complete in
 * stream order; calls that may overlap (two streams, two captured graphs)
 * need one each.  Every call can be captured into a HIP graph.
 *
 * Elements are fp32, bf16 or fp16 (policy_dtype); sums and states are fp32
 * and every stored element is rounded once, to nearest even.
 */
#ifndef POLICY_H
#define POLICY_H

#include <stdint.h>

#include "rollout.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { POLICY_F32 = 0, POLICY_BF16 = 1, POLICY_F16 = 2 } policy_dtype;

/* -------------------------------------------------------------- recurrence
 * For step t of row n (an episode) and channel d, with the gates
 *   RECUR_LINEAR   a_t = gate_t,           b_t = x_t
 *   RECUR_SIGMOID  a_t = sigmoid(gate_t),  b_t = (1 - a_t) x_t
 * the state is
 *   h_t = a_t m_t h_{t-1} + b_t,   h_{-1} = h0 (0 when NULL),
 *   m_t = 0 where dones[t-1][n] is not 0, else 1;  m_0 = 1,
 *   h_last = 0 where dones[L-1][n] is not 0, else h_{L-1}  (fp32, unrounded):
 * dones are a collection's, so the state that follows a finished episode is
 * zero, and a rollout cut in two gives the whole's results when the second
 * part starts from the first part's h_last.  m selects: a NaN or infinity of
 * a finished episode does not reach the next one.  Products of linear gates may
 * leave fp32's range: the states are those of the steps one by one all the same,
 * to fp32 roundings.  Of a state that sigmoid gates shrink below 2^-126 of
 * itself, what is left is lost.
 *
 * x, gate, h, dh, dx and dgate are [L][N][D] of one dtype, element (t, n, d)
 * at t * step + n * row + d with the strides given for each; the output
 * buffers' elements must be distinct.  dones is [L][N] u8, h0, h_last,
 * dh_last and dh0 are [N][D] f32, all contiguous.  Outputs must not overlap
 * inputs. */
typedef enum { RECUR_LINEAR = 0, RECUR_SIGMOID = 1 } recur_form;

typedef struct {
  int32_t steps, rows, width; /* L, N, D >= 0; L <= 2^30, N * D < 2^28 */
  int32_t dtype;              /* policy_dtype */
  int32_t form;               /* recur_form */
  int64_t x_step, x_row;      /* strides in elements */
  int64_t gate_step, gate_row;
  int64_t h_step, h_row;
  const void *x;
  const void *gate;
  const float *h0;      /* NULL: zero */
  const uint8_t *dones; /* NULL: none */
  void *h;
  float *h_last; /* NULL: not written */
  void *workspace; /* recur_workspace() bytes, 16-byte aligned (may be NULL when 0) */
  int64_t workspace_bytes;
} recur_args;

/* The gradient: from dh and dh_last (NULL: zero), with G_L = dh_last where the
 * last step is not done, else 0,
 *   d_t = dh_t + G_{t+1},   G_t = a_t m_t d_t,   dh0 = G_0,
 *   RECUR_LINEAR   dx_t = d_t,            dgate_t = d_t m_t h_{t-1}
 *   RECUR_SIGMOID  dx_t = (1 - a_t) d_t,  dgate_t = a_t (1 - a_t) d_t (m_t h_{t-1} - x_t)
 * h is the forward call's output, read in fp32 and in the linear form; the
 * sigmoid form of the 16-bit types takes the states in fp32 instead (`kept`
 * below), because a state that follows its input makes h_{t-1} - x_t a
 * difference of near numbers, which a rounded h would leave few digits of.
 * x is read only in the sigmoid form. */
typedef struct {
  int32_t steps, rows, width;
  int32_t dtype;
  int32_t form;
  int64_t x_step, x_row;
  int64_t gate_step, gate_row;
  int64_t h_step, h_row;
  int64_t dh_step, dh_row;
  int64_t dx_step, dx_row;
  int64_t dgate_step, dgate_row;
  const void *x; /* may be NULL in the linear form */
  const void *gate;
  const void *h; /* may be NULL in the sigmoid form of the 16-bit types */
  const float *h0;      /* NULL: zero */
  const uint8_t *dones; /* NULL: none */
  const void *dh;
  const float *dh_last; /* NULL: zero */
  void *dx;
  void *dgate;
  float *dh0; /* NULL: not written */
  void *workspace;
  int64_t workspace_bytes;
} recur_grad_args;

/* Workspace in bytes of recur_forward and of recur_backward for these sizes
 * (the same for both; 0 for most in fp32), or a negative ROLLOUT_E* code. */
int64_t recur_workspace(int32_t steps, int32_t rows, int32_t width, int32_t dtype);
/* The same of recur_forward_kept and recur_backward_kept. */
int64_t recur_kept_workspace(int32_t steps, int32_t rows, int32_t width, int32_t dtype);

/* L, N or D of 0 is a no-op, except that L = 0 copies h0 to h_last (and
 * dh_last to dh0).  Errors: ROLLOUT_EINVAL (NULL or misaligned buffer,
 * unknown dtype or form, a negative size or stride, workspace too small),
 * ROLLOUT_EHIP. */
int recur_forward(const recur_args *args, void *hip_stream);
int recur_backward(const recur_grad_args *args, void *hip_stream);
/* The same two for a training pass.  `kept` [ceil(L / 8)][N][D] f32 holds the
 * states that enter the steps 0, 8, 16, ... (before a done cuts them): the
 * first call writes it, the second, of the same x, gate, h0 and dones, takes
 * the states from there.  Only the sigmoid form of the 16-bit types uses it;
 * otherwise it may be NULL and the calls are the two above.  recur_backward
 * itself forms the states again, from x and gate. */
int recur_forward_kept(const recur_args *args, float *kept, void *hip_stream);
int recur_backward_kept(const recur_grad_args *args, const float *kept, void *hip_stream);

/* One step, for acting: h = a m state + b with m = 0 where resets[n] is not 0
 * (the episode ended before this step), new_state the same value unrounded.
 * x, gate, h are [N][D] with row strides; state and new_state [N][D] f32
 * contiguous, and may be the same buffer (an update in place). */
int recur_step(int32_t rows, int32_t width, int32_t dtype, int32_t form, const void *x,
               int64_t x_row, const void *gate, int64_t gate_row, const float *state,
               const uint8_t *resets, void *h, int64_t h_row, float *new_state,
               void *hip_stream);

/* --------------------------------------------------------------- embedding
 * out[i] = scale * weight[index[i]], rounded once; an index outside [0, vocab)
 * (an episode's first step has no previous action: -1) gives a row of zeros
 * and takes no part in the gradient.  weight: [vocab][width] with rows
 * weight_row elements apart; out: [count][width], rows out_row apart; index:
 * [count] of index_bytes 4 (i32) or 8 (i64).  The gradient is dense:
 *   dweight[v] = scale * sum of dout[i] over the i with index[i] == v,
 * summed in fp32 in ascending order of i within fixed pieces that depend on
 * the indices and sizes alone (results are deterministic), rounded once; rows
 * without an index are zero.  vocab and count are at most 2^31 - 2, width
 * at most 2^24.  dweight must not overlap dout or index. */
int embed_forward(int32_t dtype, const void *weight, int64_t vocab, int32_t width,
                  int64_t weight_row, const void *index, int32_t index_bytes, int64_t count,
                  float scale, void *out, int64_t out_row, void *hip_stream);
/* Workspace in bytes of embed_backward, or a negative ROLLOUT_E* code. */
int64_t embed_workspace(int32_t dtype, int64_t vocab, int32_t width, int64_t count);
/* count = 0 clears dweight.  Errors of both: ROLLOUT_EINVAL (NULL or
 * misaligned buffer, unknown dtype or index size, negative or too large a
 * size, rows closer than width (a row stride of 0 repeats one row of dout),
 * workspace too small), ROLLOUT_EHIP. */
int embed_backward(int32_t dtype, const void *dout, int64_t dout_row, const void *index,
                   int32_t index_bytes, int64_t count, int64_t vocab, int32_t width, float scale,
                   void *dweight, int64_t dweight_row, void *workspace, int64_t workspace_bytes,
                   void *hip_stream);

/* ------------------------------------------------------------------ logits
 * With c = the times token v occurs among the first history_len[r] (all
 * history_width when NULL; clamped into 0 .. history_width) entries of row
 * r's history, entries outside [0, vocab) not counted, and z = logits[r][v]:
 *   z = c > 0 ? (z > 0 ? z / repetition : z * repetition) : z
 *   z = z - (c > 0 ? presence : 0) - frequency * c
 *   z = z + bias[v]
 *   out[r][v] = allowed(r, v) ? z : -infinity,
 * evaluated in fp32, rounded once.  A row with nothing allowed is all
 * -infinity.  What a masked place holds (NaN included) does not matter.
 * The gradient: dlogits = allowed ? dout * (c > 0 ? (z > 0 ? 1 / repetition :
 * repetition) : 1) : 0 and dbias[v] = the sum of dout over the rows that
 * allow v, in fp32, in a fixed order.
 *
 * The penalties are per row where the _rows array [rows] f32 is given, else
 * the scalar for every row.  repetition must be positive.  The mask is
 *   LOGITS_MASK_BYTES  [mask_count][vocab] u8, rows mask_row bytes apart,
 *                      not 0 = allowed
 *   LOGITS_MASK_BITS   [mask_count][ceil(vocab / 32)] u32, rows mask_row words
 *                      apart, bit v % 32 of word v / 32 set = allowed
 * and row r uses mask row mask_rows[r] (a value outside [0, mask_count) allows
 * everything) or, where mask_rows is NULL, r (mask_count = rows) or 0
 * (mask_count = 1).  out may be logits itself (same rows, same stride), and
 * dlogits may be dout. */
typedef enum { LOGITS_MASK_NONE = 0, LOGITS_MASK_BYTES = 1, LOGITS_MASK_BITS = 2 } logits_mask;

typedef struct {
  int64_t rows;         /* R >= 0 */
  int32_t vocab;        /* V, 0 .. 2^24 */
  int32_t dtype;        /* policy_dtype of logits, out, dout, dlogits */
  const void *logits;   /* [R][V], rows logits_row elements apart */
  int64_t logits_row;
  const float *bias;    /* NULL: none; rows bias_row apart (0: one for all) */
  int64_t bias_row;
  const int32_t *history; /* NULL: none; [R][history_width], rows history_row apart */
  int64_t history_row;
  const int32_t *history_len;  /* NULL: all of the width */
  int32_t history_width;
  int32_t mask_kind;    /* logits_mask */
  float repetition, presence, frequency; /* 1, 0, 0: no penalty */
  const float *repetition_rows, *presence_rows, *frequency_rows; /* NULL: the scalars */
  const void *mask;
  int64_t mask_row, mask_count;
  const int32_t *mask_rows; /* NULL: row r, or 0 where mask_count is 1 */
} logits_args;

/* Errors: ROLLOUT_EINVAL (NULL or misaligned buffer, unknown dtype or mask
 * kind, a negative or too large a size, rows closer than their width, a scalar repetition
 * that is not positive and finite, mask_count neither 1 nor rows without
 * mask_rows, workspace too small), ROLLOUT_EHIP. */
int logits_forward(const logits_args *args, void *out, int64_t out_row, void *hip_stream);
/* Workspace in bytes of logits_backward with dbias (none is needed without). */
int64_t logits_workspace(int64_t rows, int32_t vocab);
/* dlogits or dbias [vocab] may be NULL (not computed); of args, the bias and
 * the presence and frequency penalties are not read, and the logits only
 * with a history and a repetition other than the scalar 1. */
int logits_backward(const logits_args *args, const void *dout, int64_t dout_row, void *dlogits,
                    int64_t dlogits_row, float *dbias, void *workspace, int64_t workspace_bytes,
                    void *hip_stream);

#ifdef __cplusplus
}
#endif
#endif
