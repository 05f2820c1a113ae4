// Host-side interface of the kernels of a residual block (conv.hip, scan.hip,
// scan_grad.hip, norm.hip, drop.hip, sums.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/block.h"

namespace rl {

// Sets the calling thread's rollout_last_error() text; returns `code`.
int set_error(int code, const char* text);

hipError_t conv_forward_launch(const conv_args& a, hipStream_t stream);
int64_t conv_workspace_bytes(int32_t L, int32_t N, int32_t D, int32_t W, int32_t dtype);
hipError_t conv_backward_launch(const conv_grad_args& a, hipStream_t stream);
hipError_t conv_step_launch(int32_t N, int32_t D, int32_t W, int32_t dtype, int32_t activation,
                            const void* x, int64_t x_row, const float* weight, const float* bias,
                            const void* state, const uint8_t* resets, void* y, int64_t y_row,
                            void* new_state, hipStream_t stream);

int64_t scan_kept_floats(int32_t L, int32_t N, int32_t D, int32_t S, int32_t G);
int64_t scan_workspace_bytes(int32_t L, int32_t N, int32_t D, int32_t S, int32_t G);
int64_t scan_grad_workspace_bytes(int32_t L, int32_t N, int32_t D, int32_t S, int32_t G);
hipError_t scan_forward_launch(const scan_args& a, hipStream_t stream);
hipError_t scan_backward_launch(const scan_grad_args& a, hipStream_t stream);
hipError_t scan_step_launch(const scan_args& a, hipStream_t stream);

hipError_t norm_forward_launch(const norm_args& a, void* stream_out, int64_t stream_row,
                               void* normed, int64_t normed_row, float* stats, hipStream_t stream);
int64_t norm_workspace_bytes(int64_t R, int32_t D, int32_t dtype);
hipError_t norm_backward_launch(const norm_grad_args& a, hipStream_t stream);

hipError_t drop_forward_launch(int32_t dtype, const void* x, int64_t count, float p, uint64_t seed,
                               const uint64_t* seed_at, uint32_t offset, void* out,
                               hipStream_t stream);

// out[c] = sum of the `rows` rows of x [rows][columns] (f32), in an order fixed
// by the two sizes.  Output k takes the columns from end[k - 1] to end[k] (NULL:
// not wanted).  scratch: sums_floats() floats.
struct SumsOut {
  float* out[3];
  int32_t end[3];
};
int64_t sums_floats(int64_t rows, int32_t columns);
hipError_t sums_launch(const float* x, int64_t rows, int32_t columns, float* scratch,
                       const SumsOut& out, hipStream_t stream);
// bytes (a multiple of 2) of src, or zeros where src is NULL, to dst.
hipError_t copy_or_clear_launch(const void* src, void* dst, int64_t bytes, hipStream_t stream);

}  // namespace rl
