/*
 * policy.h -- C ABI of the operators of a policy with memory in librollout.so
 * (gfx950), from the previous action to the next action's logits:
 *   recur_*   gated linear recurrence over a rollout, its gradient, its step
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
 * a finished episode does not reach the next one.
 *
 * x, gate, h, dh, dx and dgate are [L][N][D] of one dtype, element (t, n, d)
 * at t * step + n * row + d with the strides given for each; the output
 * buffers' elements must be distinct.  dones is [L][N] u8, h0, h_last,
 * dh_last and dh0 are [N][D] f32, all contiguous.  Outputs must not overlap
 * inputs. */
typedef enum { RECUR_LINEAR = 0, RECUR_SIGMOID = 1 } recur_form;

typedef struct {
  int32_t steps, rows, width; /* L, N, D >= 0; N * D < 2^31 */
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
 * h is the forward call's output (in its dtype).  x is read only in the
 * sigmoid form. */
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
  const void *h;
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
 * (the same for both; 0 for most), or a negative ROLLOUT_E* code. */
int64_t recur_workspace(int32_t steps, int32_t rows, int32_t width, int32_t dtype);

/* L, N or D of 0 is a no-op, except that L = 0 copies h0 to h_last (and
 * dh_last to dh0).  Errors: ROLLOUT_EINVAL (NULL or misaligned buffer,
 * unknown dtype or form, a negative size or stride, workspace too small),
 * ROLLOUT_EHIP. */
int recur_forward(const recur_args *args, void *hip_stream);
int recur_backward(const recur_grad_args *args, void *hip_stream);

/* One step, for acting: h = a m state + b with m = 0 where resets[n] is not 0
 * (the episode ended before this step), new_state the same value unrounded.
 * x, gate, h are [N][D] with row strides; state and new_state [N][D] f32
 * contiguous, and may be the same buffer (an update in place). */
int recur_step(int32_t rows, int32_t width, int32_t dtype, int32_t form, const void *x,
               int64_t x_row, const void *gate, int64_t gate_row, const float *state,
               const uint8_t *resets, void *h, int64_t h_row, float *new_state,
               void *hip_stream);

#ifdef __cplusplus
}
#endif
#endif
