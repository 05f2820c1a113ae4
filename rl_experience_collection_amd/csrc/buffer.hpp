// Rows addressed through buffer resources.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "elem.hpp"

namespace rl {

// Access to a row whose address and length the wave shares.  The hardware
// drops what lies past the length: lanes without a channel and steps past the
// end (length 0) read 0 and write nothing, with no branch and no clamping.
typedef uint32_t words4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_of(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00027000);
}
template <class T>
__device__ __forceinline__ typename T::raw row_load(const void* p, uint32_t bytes, uint32_t at) {
  if constexpr (T::kBytes == 4)
    return __builtin_amdgcn_raw_buffer_load_b32(row_of(p, bytes), at, 0, 0);
  else
    return __builtin_amdgcn_raw_buffer_load_b16(row_of(p, bytes), at, 0, 0);
}
template <class T>
__device__ __forceinline__ void row_store(void* p, uint32_t bytes, uint32_t at, float x) {
  if constexpr (T::kBytes == 4)
    __builtin_amdgcn_raw_buffer_store_b32(T::narrow(x), row_of(p, bytes), at, 0, 0);
  else
    __builtin_amdgcn_raw_buffer_store_b16(T::narrow(x), row_of(p, bytes), at, 0, 0);
}

// A wave waits for its loads by the number of accesses it has issued since, the
// least that any way to that point has.  In a loop that loads
// for its next turn and then stores, the loads before the loop have no stores
// after them: without n stores to a row of no length there, every turn would
// wait for the stores of the one before.
__device__ __forceinline__ void no_stores(const void* p, int n) {
#pragma unroll
  for (int i = 0; i < n; ++i) __builtin_amdgcn_raw_buffer_store_b32(i, row_of(p, 0), 256 * i, 0, 0);
}

}  // namespace rl
