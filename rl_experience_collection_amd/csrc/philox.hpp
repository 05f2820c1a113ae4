// Dropout's draws (include/block.h, drop_forward).
#pragma once

#include "device.hpp"

namespace rl {

constexpr uint32_t kDropWord = 0x44524f50u;

// What a dropped element compares with, and the scale of what is kept.
struct DropRule {
  uint32_t drop;  // of 65536
  float scale;
  uint64_t seed;
  const uint64_t* seed_at;
  uint32_t offset;
};
inline DropRule drop_rule(float p, uint64_t seed, const uint64_t* seed_at, uint32_t offset) {
  const uint32_t drop = (uint32_t)((double)p * 65536.0 + 0.5);
  return DropRule{drop, drop < 65536 ? (float)(65536.0 / (65536.0 - drop)) : 0.0f, seed, seed_at, offset};
}

// The draws of the elements 8 b .. 8 b + 7, 16 bits each, the first lowest.
__device__ __forceinline__ uint4 drop_draws(const DropRule& r, uint64_t seed, uint64_t b) {
  return philox10(make_uint4((uint32_t)b, (uint32_t)(b >> 32), r.offset, kDropWord), (uint32_t)seed,
                  (uint32_t)(seed >> 32));
}
__device__ __forceinline__ uint32_t draw_of(uint4 d, int i) {
  const uint32_t w = i < 2 ? d.x : i < 4 ? d.y : i < 6 ? d.z : d.w;
  return i & 1 ? w >> 16 : w & 0xffffu;
}

}  // namespace rl
