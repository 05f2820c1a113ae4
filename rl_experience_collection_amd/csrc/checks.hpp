// What the C entry points check of their arguments, and how they report it.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>

#include "elem.hpp"
#include "policy.hpp"

namespace rl {

inline int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return set_error(code, buf);
}

inline int launched(hipError_t e, const char* what) {
  return e == hipSuccess ? ROLLOUT_OK : fail(ROLLOUT_EHIP, "%s: %s", what, hipGetErrorString(e));
}

inline bool known_dtype(int32_t d) { return d == POLICY_F32 || d == POLICY_BF16 || d == POLICY_F16; }
inline size_t element_bytes(int32_t d) { return d == POLICY_F32 ? 4 : 2; }

// A buffer of elements: not NULL and aligned to its element.
inline int check_buffer(const char* who, const char* name, const void* p, size_t bytes) {
  if (!p) return fail(ROLLOUT_EINVAL, "%s: %s is NULL", who, name);
  if (!aligned_to(p, bytes))
    return fail(ROLLOUT_EINVAL, "%s: %s is not aligned to its %zu-byte elements", who, name, bytes);
  return ROLLOUT_OK;
}
// The same where NULL is allowed.
inline int check_optional(const char* who, const char* name, const void* p, size_t bytes) {
  return p ? check_buffer(who, name, p, bytes) : ROLLOUT_OK;
}

#define RL_CHECK(call)   \
  do {                   \
    const int _rc = (call); \
    if (_rc) return _rc; \
  } while (0)

inline int check_strides(const char* who, const char* name, int64_t step, int64_t row) {
  if (step < 0 || row < 0)
    return fail(ROLLOUT_EINVAL, "%s: negative stride of %s (%lld, %lld)", who, name, (long long)step,
                (long long)row);
  return ROLLOUT_OK;
}

inline int check_workspace(const char* who, int64_t need, const void* workspace, int64_t bytes) {
  if (need == 0) return ROLLOUT_OK;
  if (!workspace || bytes < need)
    return fail(ROLLOUT_EINVAL, "%s: workspace of %lld bytes needed, %lld given", who,
                (long long)need, workspace ? (long long)bytes : 0LL);
  return check_buffer(who, "workspace", workspace, 16);
}

// Rows of at least `width` elements, one after another.
inline int check_rows(const char* who, const char* name, int64_t row, int64_t width) {
  if (row < width)
    return fail(ROLLOUT_EINVAL, "%s: rows of %s are %lld apart, closer than their width %lld", who,
                name, (long long)row, (long long)width);
  return ROLLOUT_OK;
}

}  // namespace rl
