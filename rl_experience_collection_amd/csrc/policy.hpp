// Host-side interface of the policy operators' kernels (embed.hip,
// recur.hip, logits.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/policy.h"

namespace rl {

// Sets the calling thread's rollout_last_error() text; returns `code`.
int set_error(int code, const char* text);

// Whether the gradient takes the states from `kept`, not from h.
bool recur_keeps(int32_t dtype, int32_t form);
int64_t recur_kept_floats(int32_t L, int32_t N, int32_t D);
// The chained scans' words; without kept states the gradient's workspace
// holds those as well, first.
int64_t recur_chain_bytes(int32_t L, int32_t N, int32_t D);
// kept: NULL where they are not wanted.
hipError_t recur_forward_launch(const recur_args& a, float* kept, hipStream_t stream);
hipError_t recur_backward_launch(const recur_grad_args& a, const float* kept, hipStream_t stream);
hipError_t recur_step_launch(int32_t N, int32_t D, int32_t dtype, int32_t form, const void* x,
                             int64_t x_row, const void* gate, int64_t gate_row,
                             const float* state, const uint8_t* resets, void* h, int64_t h_row,
                             float* new_state, hipStream_t stream);

struct EmbedForward {
  const void* weight;
  const void* index;
  void* out;
  int64_t vocab, count, weight_row, out_row;
  int32_t dtype, width, index_bytes;
  float scale;
};
struct EmbedBackward {
  const void* dout;
  const void* index;
  void* dweight;
  void* workspace;
  int64_t vocab, count, dout_row, dweight_row;
  int32_t dtype, width, index_bytes;
  float scale;
};
hipError_t embed_forward_launch(const EmbedForward& a, hipStream_t stream);
int64_t embed_workspace_bytes(int32_t dtype, int64_t vocab, int32_t width, int64_t count);
hipError_t embed_backward_launch(const EmbedBackward& a, hipStream_t stream);

hipError_t logits_forward_launch(const logits_args& a, void* out, int64_t out_row,
                                 hipStream_t stream);
// Whether the gradient needs the logits: only a repetition penalty scales it.
bool logits_gradient_reads_logits(const logits_args& a);
int64_t logits_workspace_bytes(int64_t rows, int32_t vocab);
hipError_t logits_backward_launch(const logits_args& a, const void* dout, int64_t dout_row,
                                  void* dlogits, int64_t dlogits_row, float* dbias,
                                  void* workspace, hipStream_t stream);

}  // namespace rl
