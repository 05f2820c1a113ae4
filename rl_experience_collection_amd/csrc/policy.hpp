// Host-side interface of the policy operators' kernels (recur.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/policy.h"

namespace rl {

// Sets the calling thread's rollout_last_error() text; returns `code`.
int set_error(int code, const char* text);

int64_t recur_workspace_bytes(int32_t L, int32_t N, int32_t D, int32_t dtype);
hipError_t recur_forward_launch(const recur_args& a, hipStream_t stream);
hipError_t recur_backward_launch(const recur_grad_args& a, hipStream_t stream);
hipError_t recur_step_launch(int32_t N, int32_t D, int32_t dtype, int32_t form, const void* x,
                             int64_t x_row, const void* gate, int64_t gate_row,
                             const float* state, const uint8_t* resets, void* h, int64_t h_row,
                             float* new_state, hipStream_t stream);

}  // namespace rl
