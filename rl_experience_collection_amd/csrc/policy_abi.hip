// C ABI of the policy operators (include/policy.h): argument checks, then
// the launches.  Nothing is allocated and nothing is kept between calls.
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>

#include "elem.hpp"
#include "policy.hpp"

namespace {

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return rl::set_error(code, buf);
}

int launched(hipError_t e, const char* what) {
  return e == hipSuccess ? ROLLOUT_OK : fail(ROLLOUT_EHIP, "%s: %s", what, hipGetErrorString(e));
}

bool known_dtype(int32_t d) { return d == POLICY_F32 || d == POLICY_BF16 || d == POLICY_F16; }
size_t element_bytes(int32_t d) { return d == POLICY_F32 ? 4 : 2; }

// A buffer of elements: not NULL and aligned to its element.
int check_buffer(const char* who, const char* name, const void* p, size_t bytes) {
  if (!p) return fail(ROLLOUT_EINVAL, "%s: %s is NULL", who, name);
  if (!rl::aligned_to(p, bytes))
    return fail(ROLLOUT_EINVAL, "%s: %s is not aligned to its %zu-byte elements", who, name, bytes);
  return ROLLOUT_OK;
}
// The same where NULL is allowed.
int check_optional(const char* who, const char* name, const void* p, size_t bytes) {
  return p ? check_buffer(who, name, p, bytes) : ROLLOUT_OK;
}

#define RL_CHECK(call)   \
  do {                   \
    const int _rc = (call); \
    if (_rc) return _rc; \
  } while (0)

int check_recur_sizes(const char* who, int32_t steps, int32_t rows, int32_t width, int32_t dtype) {
  if (steps < 0 || rows < 0 || width < 0)
    return fail(ROLLOUT_EINVAL, "%s: negative size (steps %d, rows %d, width %d)", who, steps, rows,
                width);
  if ((int64_t)rows * width >= (int64_t)1 << 31)
    return fail(ROLLOUT_EINVAL, "%s: rows * width must be below 2^31 (got %d * %d)", who, rows, width);
  if (!known_dtype(dtype)) return fail(ROLLOUT_EINVAL, "%s: unknown dtype %d", who, dtype);
  return ROLLOUT_OK;
}

int check_form(const char* who, int32_t form) {
  if (form != RECUR_LINEAR && form != RECUR_SIGMOID)
    return fail(ROLLOUT_EINVAL, "%s: unknown form %d", who, form);
  return ROLLOUT_OK;
}

int check_strides(const char* who, const char* name, int64_t step, int64_t row) {
  if (step < 0 || row < 0)
    return fail(ROLLOUT_EINVAL, "%s: negative stride of %s (%lld, %lld)", who, name, (long long)step,
                (long long)row);
  return ROLLOUT_OK;
}

int check_recur_workspace(const char* who, int32_t steps, int32_t rows, int32_t width, int32_t dtype,
                          const void* workspace, int64_t bytes) {
  const int64_t need = rl::recur_workspace_bytes(steps, rows, width, dtype);
  if (need == 0) return ROLLOUT_OK;
  if (!workspace || bytes < need)
    return fail(ROLLOUT_EINVAL, "%s: workspace of %lld bytes needed, %lld given", who,
                (long long)need, workspace ? (long long)bytes : 0LL);
  return check_buffer(who, "workspace", workspace, 16);
}

}  // namespace

extern "C" {

int64_t recur_workspace(int32_t steps, int32_t rows, int32_t width, int32_t dtype) {
  RL_CHECK(check_recur_sizes("recur_workspace", steps, rows, width, dtype));
  return rl::recur_workspace_bytes(steps, rows, width, dtype);
}

int recur_forward(const recur_args* a, void* hip_stream) {
  const char* who = "recur_forward";
  if (!a) return fail(ROLLOUT_EINVAL, "%s: arguments are NULL", who);
  RL_CHECK(check_recur_sizes(who, a->steps, a->rows, a->width, a->dtype));
  RL_CHECK(check_form(who, a->form));
  if (a->rows == 0 || a->width == 0) return ROLLOUT_OK;
  RL_CHECK(check_optional(who, "h0", a->h0, 4));
  RL_CHECK(check_optional(who, "h_last", a->h_last, 4));
  if (a->steps > 0) {
    const size_t eb = element_bytes(a->dtype);
    RL_CHECK(check_strides(who, "x", a->x_step, a->x_row));
    RL_CHECK(check_strides(who, "gate", a->gate_step, a->gate_row));
    RL_CHECK(check_strides(who, "h", a->h_step, a->h_row));
    RL_CHECK(check_buffer(who, "x", a->x, eb));
    RL_CHECK(check_buffer(who, "gate", a->gate, eb));
    RL_CHECK(check_buffer(who, "h", a->h, eb));
    RL_CHECK(check_recur_workspace(who, a->steps, a->rows, a->width, a->dtype, a->workspace,
                                   a->workspace_bytes));
  }
  return launched(rl::recur_forward_launch(*a, static_cast<hipStream_t>(hip_stream)), who);
}

int recur_backward(const recur_grad_args* a, void* hip_stream) {
  const char* who = "recur_backward";
  if (!a) return fail(ROLLOUT_EINVAL, "%s: arguments are NULL", who);
  RL_CHECK(check_recur_sizes(who, a->steps, a->rows, a->width, a->dtype));
  RL_CHECK(check_form(who, a->form));
  if (a->rows == 0 || a->width == 0) return ROLLOUT_OK;
  RL_CHECK(check_optional(who, "h0", a->h0, 4));
  RL_CHECK(check_optional(who, "dh_last", a->dh_last, 4));
  RL_CHECK(check_optional(who, "dh0", a->dh0, 4));
  if (a->steps > 0) {
    const size_t eb = element_bytes(a->dtype);
    if (a->form == RECUR_SIGMOID) {
      RL_CHECK(check_strides(who, "x", a->x_step, a->x_row));
      RL_CHECK(check_buffer(who, "x", a->x, eb));
    }
    RL_CHECK(check_strides(who, "gate", a->gate_step, a->gate_row));
    RL_CHECK(check_strides(who, "h", a->h_step, a->h_row));
    RL_CHECK(check_strides(who, "dh", a->dh_step, a->dh_row));
    RL_CHECK(check_strides(who, "dx", a->dx_step, a->dx_row));
    RL_CHECK(check_strides(who, "dgate", a->dgate_step, a->dgate_row));
    RL_CHECK(check_buffer(who, "gate", a->gate, eb));
    RL_CHECK(check_buffer(who, "h", a->h, eb));
    RL_CHECK(check_buffer(who, "dh", a->dh, eb));
    RL_CHECK(check_buffer(who, "dx", a->dx, eb));
    RL_CHECK(check_buffer(who, "dgate", a->dgate, eb));
    RL_CHECK(check_recur_workspace(who, a->steps, a->rows, a->width, a->dtype, a->workspace,
                                   a->workspace_bytes));
  }
  return launched(rl::recur_backward_launch(*a, static_cast<hipStream_t>(hip_stream)), who);
}

int recur_step(int32_t rows, int32_t width, int32_t dtype, int32_t form, const void* x,
               int64_t x_row, const void* gate, int64_t gate_row, const float* state,
               const uint8_t* resets, void* h, int64_t h_row, float* new_state, void* hip_stream) {
  const char* who = "recur_step";
  RL_CHECK(check_recur_sizes(who, 1, rows, width, dtype));
  RL_CHECK(check_form(who, form));
  if (rows == 0 || width == 0) return ROLLOUT_OK;
  const size_t eb = element_bytes(dtype);
  RL_CHECK(check_strides(who, "x", 0, x_row));
  RL_CHECK(check_strides(who, "gate", 0, gate_row));
  RL_CHECK(check_strides(who, "h", 0, h_row));
  RL_CHECK(check_buffer(who, "x", x, eb));
  RL_CHECK(check_buffer(who, "gate", gate, eb));
  RL_CHECK(check_buffer(who, "state", state, 4));
  RL_CHECK(check_buffer(who, "h", h, eb));
  RL_CHECK(check_buffer(who, "new_state", new_state, 4));
  return launched(rl::recur_step_launch(rows, width, dtype, form, x, x_row, gate, gate_row, state,
                                        resets, h, h_row, new_state,
                                        static_cast<hipStream_t>(hip_stream)),
                  who);
}

}  // extern "C"
