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

__device__ __forceinline__ uint64_t product(uint32_t a, uint32_t b) {
  uint64_t p, carry;
  asm("v_mad_u64_u32 %0, %1, %2, %3, 0" : "=v"(p), "=s"(carry) : "v"(a), "s"(b));
  return p;
}

// Philox4x32-10 as in device.hpp, each product one 64-bit multiply-add: two
// 32-bit ones, for its halves, take twice the time (2.4 ps an evaluation over
// the whole chip, 1.7 so).
__device__ __forceinline__ uint4 philox10_wide(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = product(c.x, 0xD2511F53u), p1 = product(c.z, 0xCD9E8D57u);
    c = make_uint4((uint32_t)(p1 >> 32) ^ c.y ^ k0, (uint32_t)p1, (uint32_t)(p0 >> 32) ^ c.w ^ k1, (uint32_t)p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

// The draws of the elements 8 b .. 8 b + 7, 16 bits each, the first lowest.
__device__ __forceinline__ uint4 drop_draws(const DropRule& r, uint64_t seed, uint64_t b) {
  return philox10_wide(make_uint4((uint32_t)b, (uint32_t)(b >> 32), r.offset, kDropWord), (uint32_t)seed,
                       (uint32_t)(seed >> 32));
}
__device__ __forceinline__ uint32_t draw_of(uint4 d, int i) {
  const uint32_t w = i < 2 ? d.x : i < 4 ? d.y : i < 6 ? d.z : d.w;
  return i & 1 ? w >> 16 : w & 0xffffu;
}

}  // namespace rl
