/*
 * block.h -- C ABI of the operators of a residual block with a selective
 * memory in librollout.so (gfx950), over the [L][N] buffers of a collection:
 *   conv_*  short causal convolution, its gradient, its single step
 *   scan_*  selective state space scan, its gradient, its single step
 *   norm_*  norms after and before a block, its gate, residual and dropout
 *   drop_*  dropout from a counter, no mask stored
 * Same conventions as policy.h: DEVICE buffers owned by the caller, the
 * caller's stream and workspace, ROLLOUT_OK or a negative ROLLOUT_E* code
 * with the message in rollout_last_error(), checks on the host before
 * anything is enqueued, nothing allocated or kept, every call can be captured
 * into a HIP graph.  Elements are fp32, bf16 or fp16 (policy_dtype);
 * parameters, states and sums are fp32 and every stored element is rounded
 * once, to nearest even.  Outputs must not overlap inputs or one another
 * except where stated.
 */
#ifndef BLOCK_H
#define BLOCK_H

#include <stdint.h>

#include "policy.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { BLOCK_NONE = 0, BLOCK_SIGMOID = 1, BLOCK_SILU = 2 } block_activation;

/* ------------------------------------------------------------- convolution
 * For step t of row n (an episode) and channel d, with W taps,
 *   p_t = bias[d] + sum over j < W of weight[d][j] x_{t-W+1+j},
 *   y_t = p_t (BLOCK_NONE) or p_t sigmoid(p_t) (BLOCK_SILU),
 * over the steps of t's own episode alone: an input before a done
 * (dones[t'][n] not 0 for a t' from it up to t - 1) counts as 0, whatever it
 * holds.  Steps before the first are state[n][W-1+t'] (0 when NULL), oldest
 * first, and belong to the first step's episode; new_state are the last
 * W - 1 inputs in the same way, as the step after the last finds them (0
 * where a done cuts them off), so that a rollout cut in two gives the whole's
 * results.
 *
 * x, y, dy and dx are [L][N][D], element (t, n, d) at t * step + n * row + d;
 * state, new_state and their gradients [N][W-1][D] of the same dtype, weight
 * [D][W] and bias [D] f32, dones [L][N] u8, all contiguous.  The elements of
 * an output must be distinct. */
typedef struct {
  int32_t steps, rows, width, taps; /* L, N, D >= 0; L <= 2^30, N * D < 2^28; W 1 .. 8 */
  int32_t dtype;                    /* policy_dtype */
  int32_t activation;               /* BLOCK_NONE or BLOCK_SILU */
  int64_t x_step, x_row;            /* strides in elements */
  int64_t y_step, y_row;
  const void *x;
  const float *weight;
  const float *bias;    /* NULL: none */
  const void *state;    /* NULL: zero */
  const uint8_t *dones; /* NULL: none */
  void *y;
  void *new_state; /* NULL: not written */
} conv_args;

typedef struct {
  conv_args f; /* the forward call's; y and new_state are not used */
  int64_t dy_step, dy_row;
  int64_t dx_step, dx_row;
  const void *dy;
  const void *dnew_state; /* NULL: zero */
  void *dx;
  float *dweight; /* [D][W] */
  float *dbias;   /* [D], NULL: not written */
  void *dstate;   /* NULL: not written */
  void *workspace; /* conv_workspace() bytes, 16-byte aligned */
  int64_t workspace_bytes;
} conv_grad_args;

/* L, N or D of 0 is a no-op, except that L = 0 copies state to new_state (and
 * dnew_state to dstate) and clears the parameters' gradients.  The sums over
 * steps and rows have an order fixed by the sizes.  Errors: ROLLOUT_EINVAL
 * (NULL or misaligned buffer, unknown dtype or activation, sizes out of
 * range, negative strides, workspace too small), ROLLOUT_EHIP. */
int conv_forward(const conv_args *args, void *hip_stream);
int64_t conv_workspace(int32_t steps, int32_t rows, int32_t width, int32_t taps, int32_t dtype);
int conv_backward(const conv_grad_args *args, void *hip_stream);
/* One step, for acting: x and y [N][D] with row strides, state as above (not
 * NULL), rows with resets[n] not 0 count their state as zero.  new_state may
 * be state itself. */
int conv_step(int32_t rows, int32_t width, int32_t taps, int32_t dtype, int32_t activation,
              const void *x, int64_t x_row, const float *weight, const float *bias,
              const void *state, const uint8_t *resets, void *y, int64_t y_row, void *new_state,
              void *hip_stream);

/* -------------------------------------------------------------------- scan
 * For step t of row n, channel d (of group g = d / (D / G)) and state s, with
 *   D_t = softplus(delta_t + delta_bias[d]) (or without softplus),
 *   h_t[s] = exp(D_t rate[d][s]) m_t h_{t-1}[s] + D_t b_t[g][s] x_t,   h_{-1} = state,
 *   v_t = sum over s of c_t[g][s] h_t[s] + skip[d] x_t,
 *   y_t = v_t, or v_t gate_t sigmoid(gate_t) where a gate is given;
 *   m_t = 0 where dones[t-1][n] is not 0, else 1;  m_0 = 1,
 *   new_state = 0 where dones[L-1][n] is not 0, else h_{L-1}  (f32, unrounded).
 * m selects: a NaN or infinity of a finished episode does not reach the next
 * one.  Decays are meant to be at most 1 (rate <= 0 with softplus); of larger
 * ones, products over up to L steps must stay in fp32's range.  Where an input
 * is infinite, outputs that it reaches are infinite or NaN, not always the one
 * that the formula gives.
 *
 * x, delta, gate, y and their gradients are [L][N][D], element (t, n, d) at
 * t * step + n * row + d; b and c [L][N][G][S], element at t * step + n * row
 * + g * group + s; rate [D][S], skip and delta_bias [D], state and new_state
 * [N][D][S] are f32, dones [L][N] u8, all contiguous. */
typedef struct {
  int32_t steps, rows, width; /* L, N, D >= 0; L <= 2^30, N * D < 2^28 */
  int32_t states, groups;     /* S 1 .. 64; G >= 1 divides D */
  int32_t dtype;              /* policy_dtype */
  int32_t softplus;           /* not 0: yes */
  int64_t x_step, x_row, delta_step, delta_row, gate_step, gate_row;
  int64_t b_step, b_row, b_group, c_step, c_row, c_group;
  int64_t y_step, y_row;
  const void *x, *delta, *gate; /* gate NULL: none */
  const void *b, *c;
  const float *rate;
  const float *skip, *delta_bias, *state; /* NULL: zero */
  const uint8_t *dones;                   /* NULL: none */
  void *y;
  float *new_state; /* NULL: not written */
  /* scan_kept() floats, 16-byte aligned: the states that enter the steps 0, 8,
   * 16, ..., which the gradient starts from.  Written by the forward call
   * (NULL: not written), read by the backward call; the order is its own. */
  float *kept;
  void *workspace; /* scan_workspace() or scan_grad_workspace() bytes, 16-byte aligned */
  int64_t workspace_bytes;
} scan_args;

typedef struct {
  scan_args f; /* the forward call's; y and new_state are not used */
  int64_t dy_step, dy_row, dx_step, dx_row, ddelta_step, ddelta_row, dgate_step, dgate_row;
  int64_t db_step, db_row, db_group, dc_step, dc_row, dc_group;
  const void *dy;
  const float *dnew_state; /* NULL: zero */
  void *dx, *ddelta, *dgate; /* dgate: where there is a gate */
  void *db, *dc;
  float *drate;
  float *dskip, *ddelta_bias, *dstate; /* NULL: not written */
} scan_grad_args;

/* Floats of `kept`: about ceil(L / 8) * N * D * S (S / 2 bytes for each element
 * of x: at 16 states four times a bf16 x). */
int64_t scan_kept(int32_t steps, int32_t rows, int32_t width, int32_t states, int32_t groups);
/* Bytes (0 for most sizes), or a negative ROLLOUT_E* code. */
int64_t scan_workspace(int32_t steps, int32_t rows, int32_t width, int32_t states, int32_t groups);
int64_t scan_grad_workspace(int32_t steps, int32_t rows, int32_t width, int32_t states,
                            int32_t groups);
/* L, N or D of 0 is a no-op, except that L = 0 copies state to new_state (and
 * dnew_state to dstate), and that parameter gradients without a summand are
 * cleared (with D of 0, db and dc are left as they are).  Errors as of conv_*. */
int scan_forward(const scan_args *args, void *hip_stream);
int scan_backward(const scan_grad_args *args, void *hip_stream);
/* One step, for acting, with args->steps = 1: the step strides are not used,
 * dones is resets [N] (rows whose episode ended before this step count their
 * state as zero), state must be given, new_state may be state itself, kept
 * and workspace are not used. */
int scan_step(const scan_args *args, void *hip_stream);

/* -------------------------------------------------------------------- norm
 * Between two blocks, for each row r of D values, with
 * rms(v) = v / sqrt(mean(v^2) + eps):
 *   u = rms(branch) branch_weight  (or branch itself with branch_norm = 0)
 *   z = act(gate) u,               act: none, sigmoid or silu (without a gate z = u)
 *   z = drop(z)                    as drop_forward numbers [R][D], stream included
 *   stream = residual_scale residual + branch_scale z
 *   normed = rms(stream) weight
 * evaluated in fp32 from end to end.  Without a branch the stream is
 * residual_scale residual.  What the gate, and a branch that is not normed,
 * hold at a dropped place does not matter, nor what the gradient of the stream
 * holds there to theirs.  Weights are [D] f32 (NULL: 1).  The gate is [R][D]
 * of the rows' dtype (gate_row > 0), or one row [D] f32 for all (gate_row =
 * 0).  Rows are *_row elements apart, at least D. */
typedef struct {
  int64_t rows;  /* R >= 0 */
  int32_t width; /* D, 1 .. 8192 */
  int32_t dtype; /* policy_dtype */
  int32_t branch_norm;
  int32_t activation; /* block_activation */
  float residual_scale, branch_scale, eps;
  float drop;           /* probability, 0 .. 1 */
  uint64_t seed;        /* of the draws */
  const uint64_t *seed_at; /* not NULL: read on the device instead of seed */
  uint32_t offset;
  uint32_t pad;
  const void *residual;
  int64_t residual_row;
  const void *branch; /* NULL: none */
  int64_t branch_row;
  const void *gate; /* NULL: none */
  int64_t gate_row;
  const float *weight, *branch_weight;
} norm_args;

/* stats [R][2] f32: 1 / sqrt(mean + eps) of the branch and of the stream, for
 * the gradient (NULL: not written). */
int norm_forward(const norm_args *args, void *stream, int64_t stream_row, void *normed,
                 int64_t normed_row, float *stats, void *hip_stream);
typedef struct {
  norm_args f;
  const float *stats; /* of the forward call */
  const void *dstream; /* NULL: zero; rows dstream_row apart (0: one row for all) */
  int64_t dstream_row;
  const void *dnormed; /* NULL: zero */
  int64_t dnormed_row;
  void *dresidual; /* contiguous rows; NULL: not written */
  void *dbranch;   /* likewise, and the two below */
  void *dgate;     /* [R][D] of the dtype, or [D] f32 */
  float *dweight, *dbranch_weight; /* [D] */
  void *workspace; /* norm_workspace() bytes, 16-byte aligned */
  int64_t workspace_bytes;
} norm_grad_args;
int64_t norm_workspace(int64_t rows, int32_t width, int32_t dtype);
/* R = 0 is a no-op that clears the parameters' gradients.  Errors as of
 * conv_*. */
int norm_backward(const norm_grad_args *args, void *hip_stream);

/* ----------------------------------------------------------------- dropout
 *   out[i] = kept(i) ? scale x[i] : 0
 * with drop = floor(65536 p + 1/2), scale = 65536 / (65536 - drop) (rounded to
 * fp32) and kept(i) = h(i) >= drop, where h(i) is the 16-bit part i % 8 (low
 * halves first) of the four words of Philox4x32-10 at key seed and counter
 * (i / 8 mod 2^32, i / 2^35, offset, 0x44524f50).  The collections' draws have
 * 0 in the last word: one seed may serve both.  What a dropped place holds
 * (NaN included) does not matter.  The gradient is the same call on the
 * output's gradient.  out may be x itself. */
int drop_forward(int32_t dtype, const void *x, int64_t count, float p, uint64_t seed,
                 const uint64_t *seed_at, uint32_t offset, void *out, void *hip_stream);

#ifdef __cplusplus
}
#endif
#endif
