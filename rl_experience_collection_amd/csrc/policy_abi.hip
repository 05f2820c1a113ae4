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
  if (steps > 1 << 30)
    return fail(ROLLOUT_EINVAL, "%s: steps must be at most 2^30 (got %d)", who, steps);
  if ((int64_t)rows * width >= (int64_t)1 << 28)
    return fail(ROLLOUT_EINVAL, "%s: rows * width must be below 2^28 (got %d * %d)", who, rows, width);
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

int check_workspace(const char* who, int64_t need, const void* workspace, int64_t bytes) {
  if (need == 0) return ROLLOUT_OK;
  if (!workspace || bytes < need)
    return fail(ROLLOUT_EINVAL, "%s: workspace of %lld bytes needed, %lld given", who,
                (long long)need, workspace ? (long long)bytes : 0LL);
  return check_buffer(who, "workspace", workspace, 16);
}

// Of a gradient that forms the states again.
int64_t states_bytes(int32_t steps, int32_t rows, int32_t width) {
  return (rl::recur_kept_floats(steps, rows, width) * 4 + 255) / 256 * 256;
}

int forward_scan(const char* who, const recur_args* a, float* kept, bool keep, void* hip_stream) {
  if (!a) return fail(ROLLOUT_EINVAL, "%s: arguments are NULL", who);
  RL_CHECK(check_recur_sizes(who, a->steps, a->rows, a->width, a->dtype));
  RL_CHECK(check_form(who, a->form));
  if (a->rows == 0 || a->width == 0) return ROLLOUT_OK;
  RL_CHECK(check_optional(who, "h0", a->h0, 4));
  RL_CHECK(check_optional(who, "h_last", a->h_last, 4));
  keep = keep && rl::recur_keeps(a->dtype, a->form);
  if (a->steps > 0) {
    const size_t eb = element_bytes(a->dtype);
    RL_CHECK(check_strides(who, "x", a->x_step, a->x_row));
    RL_CHECK(check_strides(who, "gate", a->gate_step, a->gate_row));
    RL_CHECK(check_strides(who, "h", a->h_step, a->h_row));
    RL_CHECK(check_buffer(who, "x", a->x, eb));
    RL_CHECK(check_buffer(who, "gate", a->gate, eb));
    RL_CHECK(check_buffer(who, "h", a->h, eb));
    if (keep) RL_CHECK(check_buffer(who, "kept", kept, 4));
    RL_CHECK(check_workspace(who, rl::recur_chain_bytes(a->steps, a->rows, a->width), a->workspace,
                             a->workspace_bytes));
  }
  return launched(
      rl::recur_forward_launch(*a, keep ? kept : nullptr, static_cast<hipStream_t>(hip_stream)), who);
}

int backward_scan(const char* who, const recur_grad_args* a, const float* kept, bool keep,
                  void* hip_stream) {
  if (!a) return fail(ROLLOUT_EINVAL, "%s: arguments are NULL", who);
  RL_CHECK(check_recur_sizes(who, a->steps, a->rows, a->width, a->dtype));
  RL_CHECK(check_form(who, a->form));
  if (a->rows == 0 || a->width == 0) return ROLLOUT_OK;
  RL_CHECK(check_optional(who, "h0", a->h0, 4));
  RL_CHECK(check_optional(who, "dh_last", a->dh_last, 4));
  RL_CHECK(check_optional(who, "dh0", a->dh0, 4));
  const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  if (a->steps == 0) return launched(rl::recur_backward_launch(*a, nullptr, stream), who);
  const size_t eb = element_bytes(a->dtype);
  const bool states = rl::recur_keeps(a->dtype, a->form);
  if (a->form == RECUR_SIGMOID) {
    RL_CHECK(check_strides(who, "x", a->x_step, a->x_row));
    RL_CHECK(check_buffer(who, "x", a->x, eb));
  }
  RL_CHECK(check_strides(who, "gate", a->gate_step, a->gate_row));
  RL_CHECK(check_strides(who, "dh", a->dh_step, a->dh_row));
  RL_CHECK(check_strides(who, "dx", a->dx_step, a->dx_row));
  RL_CHECK(check_strides(who, "dgate", a->dgate_step, a->dgate_row));
  RL_CHECK(check_buffer(who, "gate", a->gate, eb));
  if (!states) {
    RL_CHECK(check_strides(who, "h", a->h_step, a->h_row));
    RL_CHECK(check_buffer(who, "h", a->h, eb));
  }
  RL_CHECK(check_buffer(who, "dh", a->dh, eb));
  RL_CHECK(check_buffer(who, "dx", a->dx, eb));
  RL_CHECK(check_buffer(who, "dgate", a->dgate, eb));
  if (states && keep) RL_CHECK(check_buffer(who, "kept", kept, 4));
  const int64_t chain = rl::recur_chain_bytes(a->steps, a->rows, a->width);
  const int64_t again = states && !keep ? states_bytes(a->steps, a->rows, a->width) : 0;
  RL_CHECK(check_workspace(who, again + chain, a->workspace, a->workspace_bytes));
  if (!again) return launched(rl::recur_backward_launch(*a, kept, stream), who);
  // the states once more, into the workspace
  float* own = static_cast<float*>(a->workspace);
  recur_grad_args g = *a;
  g.workspace = static_cast<char*>(a->workspace) + again;
  g.workspace_bytes = a->workspace_bytes - again;
  recur_args f{};
  f.steps = a->steps;
  f.rows = a->rows;
  f.width = a->width;
  f.dtype = a->dtype;
  f.form = a->form;
  f.x_step = a->x_step;
  f.x_row = a->x_row;
  f.gate_step = a->gate_step;
  f.gate_row = a->gate_row;
  f.x = a->x;
  f.gate = a->gate;
  f.h0 = a->h0;
  f.dones = a->dones;
  f.workspace = g.workspace;
  f.workspace_bytes = g.workspace_bytes;
  RL_CHECK(launched(rl::recur_forward_launch(f, own, stream), who));
  return launched(rl::recur_backward_launch(g, own, stream), who);
}

constexpr int32_t kMaxWidth = 1 << 24;
constexpr int64_t kMaxCount = ((int64_t)1 << 31) - 2;

int check_embed_sizes(const char* who, int32_t dtype, int64_t vocab, int32_t width, int64_t count) {
  if (!known_dtype(dtype)) return fail(ROLLOUT_EINVAL, "%s: unknown dtype %d", who, dtype);
  if (vocab < 0 || vocab > kMaxCount || count < 0 || count > kMaxCount)
    return fail(ROLLOUT_EINVAL, "%s: vocab and count must be in 0 .. 2^31 - 2 (got %lld, %lld)", who,
                (long long)vocab, (long long)count);
  if (width < 0 || width > kMaxWidth)
    return fail(ROLLOUT_EINVAL, "%s: width must be in 0 .. 2^24 (got %d)", who, width);
  return ROLLOUT_OK;
}

int check_index(const char* who, const void* index, int32_t bytes) {
  if (bytes != 4 && bytes != 8)
    return fail(ROLLOUT_EINVAL, "%s: index_bytes must be 4 or 8 (got %d)", who, bytes);
  return check_buffer(who, "index", index, (size_t)bytes);
}

// Rows of at least `width` elements, one after another.
int check_rows(const char* who, const char* name, int64_t row, int64_t width) {
  if (row < width)
    return fail(ROLLOUT_EINVAL, "%s: rows of %s are %lld apart, closer than their width %lld", who,
                name, (long long)row, (long long)width);
  return ROLLOUT_OK;
}

int check_logits(const char* who, const logits_args* a, bool read_logits) {
  if (!a) return fail(ROLLOUT_EINVAL, "%s: arguments are NULL", who);
  if (!known_dtype(a->dtype)) return fail(ROLLOUT_EINVAL, "%s: unknown dtype %d", who, a->dtype);
  if (a->rows < 0 || a->vocab < 0 || a->vocab > kMaxWidth || a->history_width < 0)
    return fail(ROLLOUT_EINVAL,
                "%s: rows and history_width must not be negative, vocab in 0 .. 2^24 (got %lld, %d, %d)",
                who, (long long)a->rows, a->history_width, a->vocab);
  if (!(a->repetition > 0.0f && a->repetition <= 3.402823466e38f))
    return fail(ROLLOUT_EINVAL, "%s: repetition must be positive and finite (got %g)", who,
                (double)a->repetition);
  if (a->mask_kind != LOGITS_MASK_NONE && a->mask_kind != LOGITS_MASK_BYTES &&
      a->mask_kind != LOGITS_MASK_BITS)
    return fail(ROLLOUT_EINVAL, "%s: unknown mask_kind %d", who, a->mask_kind);
  if (a->rows == 0 || a->vocab == 0) return ROLLOUT_OK;
  if (read_logits) {
    RL_CHECK(check_buffer(who, "logits", a->logits, element_bytes(a->dtype)));
    RL_CHECK(check_rows(who, "logits", a->logits_row, a->vocab));
  }
  RL_CHECK(check_optional(who, "bias", a->bias, 4));
  if (a->bias && a->bias_row != 0) RL_CHECK(check_rows(who, "bias", a->bias_row, a->vocab));
  RL_CHECK(check_optional(who, "history", a->history, 4));
  if (a->history && a->history_row < 0)
    return fail(ROLLOUT_EINVAL, "%s: negative stride of history", who);
  RL_CHECK(check_optional(who, "history_len", a->history_len, 4));
  RL_CHECK(check_optional(who, "repetition_rows", a->repetition_rows, 4));
  RL_CHECK(check_optional(who, "presence_rows", a->presence_rows, 4));
  RL_CHECK(check_optional(who, "frequency_rows", a->frequency_rows, 4));
  if (a->mask_kind != LOGITS_MASK_NONE) {
    const bool bits = a->mask_kind == LOGITS_MASK_BITS;
    if (a->mask_count < 0 || a->mask_count > kMaxCount)
      return fail(ROLLOUT_EINVAL, "%s: mask_count %lld out of range", who, (long long)a->mask_count);
    RL_CHECK(check_optional(who, "mask_rows", a->mask_rows, 4));
    if (!a->mask_rows && a->mask_count != 1 && a->mask_count != a->rows)
      return fail(ROLLOUT_EINVAL, "%s: without mask_rows the mask has 1 or %lld rows (got %lld)", who,
                  (long long)a->rows, (long long)a->mask_count);
    if (a->mask_count > 0) {
      RL_CHECK(check_buffer(who, "mask", a->mask, bits ? 4 : 1));
      if (a->mask_count > 1)
        RL_CHECK(check_rows(who, "mask", a->mask_row, bits ? (a->vocab + 31) / 32 : a->vocab));
    }
  }
  return ROLLOUT_OK;
}

}  // namespace

extern "C" {

int64_t recur_workspace(int32_t steps, int32_t rows, int32_t width, int32_t dtype) {
  RL_CHECK(check_recur_sizes("recur_workspace", steps, rows, width, dtype));
  if ((int64_t)rows * width == 0) return 0;
  return rl::recur_chain_bytes(steps, rows, width) +
         (rl::recur_keeps(dtype, RECUR_SIGMOID) ? states_bytes(steps, rows, width) : 0);
}

int64_t recur_kept_workspace(int32_t steps, int32_t rows, int32_t width, int32_t dtype) {
  RL_CHECK(check_recur_sizes("recur_kept_workspace", steps, rows, width, dtype));
  return rl::recur_chain_bytes(steps, rows, width);
}

int recur_forward(const recur_args* a, void* hip_stream) {
  return forward_scan("recur_forward", a, nullptr, false, hip_stream);
}
int recur_backward(const recur_grad_args* a, void* hip_stream) {
  return backward_scan("recur_backward", a, nullptr, false, hip_stream);
}
int recur_forward_kept(const recur_args* a, float* kept, void* hip_stream) {
  return forward_scan("recur_forward_kept", a, kept, true, hip_stream);
}
int recur_backward_kept(const recur_grad_args* a, const float* kept, void* hip_stream) {
  return backward_scan("recur_backward_kept", a, kept, true, hip_stream);
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

int embed_forward(int32_t dtype, const void* weight, int64_t vocab, int32_t width,
                  int64_t weight_row, const void* index, int32_t index_bytes, int64_t count,
                  float scale, void* out, int64_t out_row, void* hip_stream) {
  const char* who = "embed_forward";
  RL_CHECK(check_embed_sizes(who, dtype, vocab, width, count));
  if (count == 0 || width == 0) return ROLLOUT_OK;
  const size_t eb = element_bytes(dtype);
  if (vocab > 0) {
    RL_CHECK(check_buffer(who, "weight", weight, eb));
    RL_CHECK(check_rows(who, "weight", weight_row, width));
  }
  RL_CHECK(check_index(who, index, index_bytes));
  RL_CHECK(check_buffer(who, "out", out, eb));
  RL_CHECK(check_rows(who, "out", out_row, width));
  rl::EmbedForward a{weight, index, out, vocab, count, weight_row, out_row, dtype, width, index_bytes,
                     scale};
  return launched(rl::embed_forward_launch(a, static_cast<hipStream_t>(hip_stream)), who);
}

int64_t embed_workspace(int32_t dtype, int64_t vocab, int32_t width, int64_t count) {
  RL_CHECK(check_embed_sizes("embed_workspace", dtype, vocab, width, count));
  return rl::embed_workspace_bytes(dtype, vocab, width, count);
}

int embed_backward(int32_t dtype, const void* dout, int64_t dout_row, const void* index,
                   int32_t index_bytes, int64_t count, int64_t vocab, int32_t width, float scale,
                   void* dweight, int64_t dweight_row, void* workspace, int64_t workspace_bytes,
                   void* hip_stream) {
  const char* who = "embed_backward";
  RL_CHECK(check_embed_sizes(who, dtype, vocab, width, count));
  if (vocab == 0 || width == 0) return ROLLOUT_OK;
  const size_t eb = element_bytes(dtype);
  if (count > 0) {
    RL_CHECK(check_buffer(who, "dout", dout, eb));
    if (dout_row != 0) RL_CHECK(check_rows(who, "dout", dout_row, width));
    RL_CHECK(check_index(who, index, index_bytes));
  }
  RL_CHECK(check_buffer(who, "dweight", dweight, eb));
  RL_CHECK(check_rows(who, "dweight", dweight_row, width));
  RL_CHECK(check_workspace(who, rl::embed_workspace_bytes(dtype, vocab, width, count), workspace,
                           workspace_bytes));
  rl::EmbedBackward a{dout, index, dweight, workspace, vocab, count, dout_row, dweight_row,
                      dtype, width, index_bytes, scale};
  return launched(rl::embed_backward_launch(a, static_cast<hipStream_t>(hip_stream)), who);
}

int logits_forward(const logits_args* a, void* out, int64_t out_row, void* hip_stream) {
  const char* who = "logits_forward";
  RL_CHECK(check_logits(who, a, true));
  if (a->rows == 0 || a->vocab == 0) return ROLLOUT_OK;
  RL_CHECK(check_buffer(who, "out", out, element_bytes(a->dtype)));
  RL_CHECK(check_rows(who, "out", out_row, a->vocab));
  return launched(rl::logits_forward_launch(*a, out, out_row, static_cast<hipStream_t>(hip_stream)),
                  who);
}

int64_t logits_workspace(int64_t rows, int32_t vocab) {
  if (rows < 0 || vocab < 0 || vocab > kMaxWidth)
    return fail(ROLLOUT_EINVAL, "logits_workspace: bad size (%lld, %d)", (long long)rows, vocab);
  return rl::logits_workspace_bytes(rows, vocab);
}

int logits_backward(const logits_args* a, const void* dout, int64_t dout_row, void* dlogits,
                    int64_t dlogits_row, float* dbias, void* workspace, int64_t workspace_bytes,
                    void* hip_stream) {
  const char* who = "logits_backward";
  RL_CHECK(check_logits(who, a, a && rl::logits_gradient_reads_logits(*a)));
  if (a->vocab == 0) return ROLLOUT_OK;
  RL_CHECK(check_optional(who, "dbias", dbias, 4));
  if (a->rows > 0) {
    const size_t eb = element_bytes(a->dtype);
    RL_CHECK(check_buffer(who, "dout", dout, eb));
    if (dout_row != 0) RL_CHECK(check_rows(who, "dout", dout_row, a->vocab));
    RL_CHECK(check_optional(who, "dlogits", dlogits, eb));
    if (dlogits) RL_CHECK(check_rows(who, "dlogits", dlogits_row, a->vocab));
    if (dbias) {
      RL_CHECK(check_workspace(who, rl::logits_workspace_bytes(a->rows, a->vocab), workspace,
                               workspace_bytes));
    }
  }
  return launched(rl::logits_backward_launch(*a, dout, dout_row, dlogits, dlogits_row, dbias,
                                             workspace, static_cast<hipStream_t>(hip_stream)),
                  who);
}

}  // extern "C"
