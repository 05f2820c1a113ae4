// C ABI of the operators of a residual block (include/block.h): argument
// checks, then the launches.  Nothing is allocated and nothing is kept
// between calls.
#include <hip/hip_runtime.h>

#include "block.hpp"
#include "checks.hpp"

using namespace rl;

namespace {

constexpr int64_t kMostColumns = (int64_t)1 << 30;  // of parameters' gradients

int check_sizes(const char* who, int32_t steps, int32_t rows, int32_t width, int32_t dtype) {
  if (steps < 0 || rows < 0 || width < 0)
    return fail(ROLLOUT_EINVAL, "%s: negative size (steps %d, rows %d, width %d)", who, steps, rows,
                width);
  if (steps > 1 << 30)
    return fail(ROLLOUT_EINVAL, "%s: steps must be at most 2^30 (got %d)", who, steps);
  if ((int64_t)rows * width >= (int64_t)1 << 28)
    return fail(ROLLOUT_EINVAL, "%s: rows * width must be below 2^28 (got %d * %d)", who, rows, width);
  if (!known_dtype(dtype)) return fail(ROLLOUT_EINVAL, "%s: unknown dtype %d", who, dtype);
  return ROLLOUT_OK;
}

int check_array(const char* who, const char* name, const void* p, int64_t step, int64_t row, size_t bytes) {
  RL_CHECK(check_strides(who, name, step, row));
  return check_buffer(who, name, p, bytes);
}

// ------------------------------------------------------------- convolution
int check_taps(const char* who, int32_t taps, int32_t activation, int32_t width) {
  if (taps < 1 || taps > 8) return fail(ROLLOUT_EINVAL, "%s: taps must be 1 to 8 (got %d)", who, taps);
  if (activation != BLOCK_NONE && activation != BLOCK_SILU)
    return fail(ROLLOUT_EINVAL, "%s: unknown activation %d", who, activation);
  if ((int64_t)width * (taps + 1) >= kMostColumns)
    return fail(ROLLOUT_EINVAL, "%s: width * (taps + 1) must be below 2^30 (got %d, %d)", who, width, taps);
  return ROLLOUT_OK;
}
int check_conv(const char* who, const conv_args& a) {
  RL_CHECK(check_sizes(who, a.steps, a.rows, a.width, a.dtype));
  RL_CHECK(check_taps(who, a.taps, a.activation, a.width));
  if (a.rows == 0 || a.width == 0) return ROLLOUT_OK;
  RL_CHECK(check_optional(who, "state", a.state, element_bytes(a.dtype)));
  if (a.steps == 0) return ROLLOUT_OK;
  RL_CHECK(check_array(who, "x", a.x, a.x_step, a.x_row, element_bytes(a.dtype)));
  RL_CHECK(check_buffer(who, "weight", a.weight, 4));
  return check_optional(who, "bias", a.bias, 4);
}

// -------------------------------------------------------------------- scan
int check_states(const char* who, int32_t width, int32_t rows, int32_t states, int32_t groups) {
  if (states < 1 || states > 64)
    return fail(ROLLOUT_EINVAL, "%s: states must be 1 to 64 (got %d)", who, states);
  if (groups < 1 || width % groups != 0)
    return fail(ROLLOUT_EINVAL, "%s: groups must divide the width (got %d of %d)", who, groups, width);
  if ((int64_t)width * (states + 2) >= kMostColumns)
    return fail(ROLLOUT_EINVAL, "%s: width * (states + 2) must be below 2^30 (got %d, %d)", who, width, states);
  // (a wave for each 64 channels of a row's group)
  const int64_t waves = (int64_t)rows * groups * ((width / groups + 63) / 64);
  if (waves > (int64_t)1 << 23)
    return fail(ROLLOUT_EINVAL, "%s: rows * groups * ceil(width / groups / 64) must be at most 2^23 (got %lld)", who,
                (long long)waves);
  return ROLLOUT_OK;
}
int check_scan_sizes(const char* who, const scan_args& a) {
  RL_CHECK(check_sizes(who, a.steps, a.rows, a.width, a.dtype));
  return check_states(who, a.width, a.rows, a.states, a.groups);
}
// What both directions and the step read.
int check_scan_inputs(const char* who, const scan_args& a) {
  const size_t eb = element_bytes(a.dtype);
  RL_CHECK(check_array(who, "x", a.x, a.x_step, a.x_row, eb));
  RL_CHECK(check_array(who, "delta", a.delta, a.delta_step, a.delta_row, eb));
  if (a.gate) RL_CHECK(check_array(who, "gate", a.gate, a.gate_step, a.gate_row, eb));
  RL_CHECK(check_array(who, "b", a.b, a.b_step, a.b_row, eb));
  RL_CHECK(check_strides(who, "b", a.b_group, 0));
  RL_CHECK(check_array(who, "c", a.c, a.c_step, a.c_row, eb));
  RL_CHECK(check_strides(who, "c", a.c_group, 0));
  RL_CHECK(check_buffer(who, "rate", a.rate, 4));
  RL_CHECK(check_optional(who, "skip", a.skip, 4));
  return check_optional(who, "delta_bias", a.delta_bias, 4);
}

// -------------------------------------------------------------------- norm
constexpr int32_t kMostWidth = 8192;

int check_norm(const char* who, const norm_args& a) {
  if (a.rows < 0) return fail(ROLLOUT_EINVAL, "%s: negative rows %lld", who, (long long)a.rows);
  if (a.width < 1 || a.width > kMostWidth)
    return fail(ROLLOUT_EINVAL, "%s: width must be 1 to %d (got %d)", who, kMostWidth, a.width);
  if (a.rows > ((int64_t)1 << 46))
    return fail(ROLLOUT_EINVAL, "%s: rows must be at most 2^46 (got %lld)", who, (long long)a.rows);
  if (!known_dtype(a.dtype)) return fail(ROLLOUT_EINVAL, "%s: unknown dtype %d", who, a.dtype);
  if (a.activation < BLOCK_NONE || a.activation > BLOCK_SILU)
    return fail(ROLLOUT_EINVAL, "%s: unknown activation %d", who, a.activation);
  if (!(a.drop >= 0.0f && a.drop <= 1.0f))
    return fail(ROLLOUT_EINVAL, "%s: drop must be 0 to 1 (got %g)", who, a.drop);
  if (!(a.eps >= 0.0f)) return fail(ROLLOUT_EINVAL, "%s: eps must not be negative (got %g)", who, a.eps);
  if (a.rows > 0 && !a.branch && (a.gate || a.branch_weight || a.drop > 0.0f))
    return fail(ROLLOUT_EINVAL, "%s: a gate, a branch_weight or dropout without a branch", who);
  if (!a.branch_norm && a.branch_weight)
    return fail(ROLLOUT_EINVAL, "%s: branch_weight without branch_norm", who);
  RL_CHECK(check_optional(who, "seed_at", a.seed_at, 8));
  RL_CHECK(check_optional(who, "weight", a.weight, 4));
  RL_CHECK(check_optional(who, "branch_weight", a.branch_weight, 4));
  if (a.rows == 0) return ROLLOUT_OK;
  const size_t eb = element_bytes(a.dtype);
  RL_CHECK(check_buffer(who, "residual", a.residual, eb));
  RL_CHECK(check_rows(who, "residual", a.residual_row, a.width));
  if (a.branch) {
    RL_CHECK(check_buffer(who, "branch", a.branch, eb));
    RL_CHECK(check_rows(who, "branch", a.branch_row, a.width));
  }
  if (a.gate) {
    RL_CHECK(check_buffer(who, "gate", a.gate, a.gate_row ? eb : 4));
    if (a.gate_row) RL_CHECK(check_rows(who, "gate", a.gate_row, a.width));
  }
  return ROLLOUT_OK;
}

}  // namespace

extern "C" {

int conv_forward(const conv_args* a, void* hip_stream) {
  const char* who = "conv_forward";
  if (!a) return fail(ROLLOUT_EINVAL, "%s: arguments are NULL", who);
  RL_CHECK(check_conv(who, *a));
  if (a->rows == 0 || a->width == 0) return ROLLOUT_OK;
  RL_CHECK(check_optional(who, "new_state", a->new_state, element_bytes(a->dtype)));
  if (a->steps > 0) RL_CHECK(check_array(who, "y", a->y, a->y_step, a->y_row, element_bytes(a->dtype)));
  return launched(rl::conv_forward_launch(*a, static_cast<hipStream_t>(hip_stream)), who);
}

int64_t conv_workspace(int32_t steps, int32_t rows, int32_t width, int32_t taps, int32_t dtype) {
  const char* who = "conv_workspace";
  RL_CHECK(check_sizes(who, steps, rows, width, dtype));
  RL_CHECK(check_taps(who, taps, BLOCK_NONE, width));
  return rl::conv_workspace_bytes(steps, rows, width, taps, dtype);
}

int conv_backward(const conv_grad_args* g, void* hip_stream) {
  const char* who = "conv_backward";
  if (!g) return fail(ROLLOUT_EINVAL, "%s: arguments are NULL", who);
  const conv_args& a = g->f;
  RL_CHECK(check_conv(who, a));
  if (a.width == 0) return ROLLOUT_OK;
  const size_t eb = element_bytes(a.dtype);
  RL_CHECK(check_buffer(who, "dweight", g->dweight, 4));
  RL_CHECK(check_optional(who, "dbias", g->dbias, 4));
  RL_CHECK(check_optional(who, "dnew_state", g->dnew_state, eb));
  RL_CHECK(check_optional(who, "dstate", g->dstate, eb));
  if (a.rows > 0 && a.steps > 0) {
    RL_CHECK(check_array(who, "dy", g->dy, g->dy_step, g->dy_row, eb));
    RL_CHECK(check_array(who, "dx", g->dx, g->dx_step, g->dx_row, eb));
    RL_CHECK(check_workspace(who, rl::conv_workspace_bytes(a.steps, a.rows, a.width, a.taps, a.dtype),
                             g->workspace, g->workspace_bytes));
  }
  return launched(rl::conv_backward_launch(*g, static_cast<hipStream_t>(hip_stream)), who);
}

int conv_step(int32_t rows, int32_t width, int32_t taps, int32_t dtype, int32_t activation,
              const void* x, int64_t x_row, const float* weight, const float* bias,
              const void* state, const uint8_t* resets, void* y, int64_t y_row, void* new_state,
              void* hip_stream) {
  const char* who = "conv_step";
  RL_CHECK(check_sizes(who, 1, rows, width, dtype));
  RL_CHECK(check_taps(who, taps, activation, width));
  if (rows == 0 || width == 0) return ROLLOUT_OK;
  const size_t eb = element_bytes(dtype);
  RL_CHECK(check_array(who, "x", x, 0, x_row, eb));
  RL_CHECK(check_buffer(who, "weight", weight, 4));
  RL_CHECK(check_optional(who, "bias", bias, 4));
  if (taps > 1) {
    RL_CHECK(check_buffer(who, "state", state, eb));
    RL_CHECK(check_buffer(who, "new_state", new_state, eb));
  }
  RL_CHECK(check_array(who, "y", y, 0, y_row, eb));
  return launched(rl::conv_step_launch(rows, width, taps, dtype, activation, x, x_row, weight, bias, state,
                                       resets, y, y_row, new_state, static_cast<hipStream_t>(hip_stream)),
                  who);
}

int64_t scan_kept(int32_t steps, int32_t rows, int32_t width, int32_t states, int32_t groups) {
  const char* who = "scan_kept";
  RL_CHECK(check_sizes(who, steps, rows, width, POLICY_F32));
  RL_CHECK(check_states(who, width, rows, states, groups));
  return rl::scan_kept_floats(steps, rows, width, states, groups);
}
int64_t scan_workspace(int32_t steps, int32_t rows, int32_t width, int32_t states, int32_t groups) {
  const char* who = "scan_workspace";
  RL_CHECK(check_sizes(who, steps, rows, width, POLICY_F32));
  RL_CHECK(check_states(who, width, rows, states, groups));
  return rl::scan_workspace_bytes(steps, rows, width, states, groups);
}
int64_t scan_grad_workspace(int32_t steps, int32_t rows, int32_t width, int32_t states, int32_t groups) {
  const char* who = "scan_grad_workspace";
  RL_CHECK(check_sizes(who, steps, rows, width, POLICY_F32));
  RL_CHECK(check_states(who, width, rows, states, groups));
  return rl::scan_grad_workspace_bytes(steps, rows, width, states, groups);
}

int scan_forward(const scan_args* a, void* hip_stream) {
  const char* who = "scan_forward";
  if (!a) return fail(ROLLOUT_EINVAL, "%s: arguments are NULL", who);
  RL_CHECK(check_scan_sizes(who, *a));
  if (a->rows == 0 || a->width == 0) return ROLLOUT_OK;
  RL_CHECK(check_optional(who, "state", a->state, 4));
  RL_CHECK(check_optional(who, "new_state", a->new_state, 4));
  if (a->steps > 0) {
    RL_CHECK(check_scan_inputs(who, *a));
    RL_CHECK(check_array(who, "y", a->y, a->y_step, a->y_row, element_bytes(a->dtype)));
    RL_CHECK(check_optional(who, "kept", a->kept, 16));
    RL_CHECK(check_workspace(who, rl::scan_workspace_bytes(a->steps, a->rows, a->width, a->states, a->groups),
                             a->workspace, a->workspace_bytes));
  }
  return launched(rl::scan_forward_launch(*a, static_cast<hipStream_t>(hip_stream)), who);
}

int scan_backward(const scan_grad_args* g, void* hip_stream) {
  const char* who = "scan_backward";
  if (!g) return fail(ROLLOUT_EINVAL, "%s: arguments are NULL", who);
  const scan_args& a = g->f;
  RL_CHECK(check_scan_sizes(who, a));
  if (a.width == 0) return ROLLOUT_OK;
  RL_CHECK(check_buffer(who, "drate", g->drate, 4));
  RL_CHECK(check_optional(who, "dskip", g->dskip, 4));
  RL_CHECK(check_optional(who, "ddelta_bias", g->ddelta_bias, 4));
  RL_CHECK(check_optional(who, "dnew_state", g->dnew_state, 4));
  RL_CHECK(check_optional(who, "dstate", g->dstate, 4));
  if (a.rows > 0 && a.steps > 0) {
    const size_t eb = element_bytes(a.dtype);
    RL_CHECK(check_scan_inputs(who, a));
    RL_CHECK(check_buffer(who, "kept", a.kept, 16));
    RL_CHECK(check_array(who, "dy", g->dy, g->dy_step, g->dy_row, eb));
    RL_CHECK(check_array(who, "dx", g->dx, g->dx_step, g->dx_row, eb));
    RL_CHECK(check_array(who, "ddelta", g->ddelta, g->ddelta_step, g->ddelta_row, eb));
    if (a.gate) RL_CHECK(check_array(who, "dgate", g->dgate, g->dgate_step, g->dgate_row, eb));
    RL_CHECK(check_array(who, "db", g->db, g->db_step, g->db_row, eb));
    RL_CHECK(check_strides(who, "db", g->db_group, 0));
    RL_CHECK(check_array(who, "dc", g->dc, g->dc_step, g->dc_row, eb));
    RL_CHECK(check_strides(who, "dc", g->dc_group, 0));
    RL_CHECK(check_workspace(who, rl::scan_grad_workspace_bytes(a.steps, a.rows, a.width, a.states, a.groups),
                             a.workspace, a.workspace_bytes));
  }
  return launched(rl::scan_backward_launch(*g, static_cast<hipStream_t>(hip_stream)), who);
}

int scan_step(const scan_args* a, void* hip_stream) {
  const char* who = "scan_step";
  if (!a) return fail(ROLLOUT_EINVAL, "%s: arguments are NULL", who);
  RL_CHECK(check_scan_sizes(who, *a));
  if (a->steps != 1) return fail(ROLLOUT_EINVAL, "%s: steps must be 1 (got %d)", who, a->steps);
  if (a->rows == 0 || a->width == 0) return ROLLOUT_OK;
  int64_t lanes = 1;
  while (4 * lanes < a->states) lanes *= 2;
  if ((int64_t)a->rows * a->width * lanes >= (int64_t)1 << 31)
    return fail(ROLLOUT_EINVAL, "%s: rows * width * ceil(states / 4) must be below 2^31", who);
  RL_CHECK(check_scan_inputs(who, *a));
  RL_CHECK(check_buffer(who, "state", a->state, 4));
  RL_CHECK(check_buffer(who, "new_state", a->new_state, 4));
  RL_CHECK(check_array(who, "y", a->y, a->y_step, a->y_row, element_bytes(a->dtype)));
  return launched(rl::scan_step_launch(*a, static_cast<hipStream_t>(hip_stream)), who);
}

int norm_forward(const norm_args* a, void* stream, int64_t stream_row, void* normed, int64_t normed_row,
                 float* stats, void* hip_stream) {
  const char* who = "norm_forward";
  if (!a) return fail(ROLLOUT_EINVAL, "%s: arguments are NULL", who);
  RL_CHECK(check_norm(who, *a));
  const size_t eb = element_bytes(a->dtype);
  if (a->rows == 0) return ROLLOUT_OK;
  RL_CHECK(check_buffer(who, "stream", stream, eb));
  RL_CHECK(check_rows(who, "stream", stream_row, a->width));
  RL_CHECK(check_buffer(who, "normed", normed, eb));
  RL_CHECK(check_rows(who, "normed", normed_row, a->width));
  RL_CHECK(check_optional(who, "stats", stats, 4));
  return launched(rl::norm_forward_launch(*a, stream, stream_row, normed, normed_row, stats,
                                          static_cast<hipStream_t>(hip_stream)),
                  who);
}

int64_t norm_workspace(int64_t rows, int32_t width, int32_t dtype) {
  if (rows < 0 || width < 1 || width > kMostWidth || !known_dtype(dtype))
    return fail(ROLLOUT_EINVAL, "norm_workspace: bad size (%lld, %d) or dtype %d", (long long)rows, width, dtype);
  return rl::norm_workspace_bytes(rows, width, dtype);
}

int norm_backward(const norm_grad_args* g, void* hip_stream) {
  const char* who = "norm_backward";
  if (!g) return fail(ROLLOUT_EINVAL, "%s: arguments are NULL", who);
  const norm_args& a = g->f;
  RL_CHECK(check_norm(who, a));
  const size_t eb = element_bytes(a.dtype);
  const bool channel = a.gate && a.gate_row == 0;
  RL_CHECK(check_optional(who, "dweight", g->dweight, 4));
  RL_CHECK(check_optional(who, "dbranch_weight", g->dbranch_weight, 4));
  RL_CHECK(check_optional(who, "dgate", g->dgate, channel ? 4 : eb));
  if (a.rows > 0) {
    RL_CHECK(check_buffer(who, "stats", g->stats, 4));
    RL_CHECK(check_optional(who, "dstream", g->dstream, eb));
    if (g->dstream && g->dstream_row != 0) RL_CHECK(check_rows(who, "dstream", g->dstream_row, a.width));
    RL_CHECK(check_optional(who, "dnormed", g->dnormed, eb));
    if (g->dnormed && g->dnormed_row != 0) RL_CHECK(check_rows(who, "dnormed", g->dnormed_row, a.width));
    RL_CHECK(check_optional(who, "dresidual", g->dresidual, eb));
    RL_CHECK(check_optional(who, "dbranch", g->dbranch, eb));
    RL_CHECK(check_workspace(who, rl::norm_workspace_bytes(a.rows, a.width, a.dtype), g->workspace,
                             g->workspace_bytes));
  }
  return launched(rl::norm_backward_launch(*g, static_cast<hipStream_t>(hip_stream)), who);
}

int drop_forward(int32_t dtype, const void* x, int64_t count, float p, uint64_t seed,
                 const uint64_t* seed_at, uint32_t offset, void* out, void* hip_stream) {
  const char* who = "drop_forward";
  if (!known_dtype(dtype)) return fail(ROLLOUT_EINVAL, "%s: unknown dtype %d", who, dtype);
  if (count < 0 || count > ((int64_t)1 << 60))
    return fail(ROLLOUT_EINVAL, "%s: bad count %lld", who, (long long)count);
  if (!(p >= 0.0f && p <= 1.0f)) return fail(ROLLOUT_EINVAL, "%s: p must be 0 to 1 (got %g)", who, p);
  RL_CHECK(check_optional(who, "seed_at", seed_at, 8));
  if (count == 0) return ROLLOUT_OK;
  RL_CHECK(check_buffer(who, "x", x, element_bytes(dtype)));
  RL_CHECK(check_buffer(who, "out", out, element_bytes(dtype)));
  return launched(rl::drop_forward_launch(dtype, x, count, p, seed, seed_at, offset, out,
                                          static_cast<hipStream_t>(hip_stream)),
                  who);
}

}  // extern "C"
