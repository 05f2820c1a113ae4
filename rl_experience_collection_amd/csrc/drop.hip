// Dropout from a counter (include/block.h).
//
// A thread draws once for eight consecutive elements: ten rounds of Philox are
// some 200 issue slots, and with 16 bits an element they stay below what
// moving the elements takes (with 32 bits, 4 elements a draw, they would not).
// No mask is stored; the gradient draws again.  1,024,001 x 129 bf16 takes 87 us,
// 6.1 TB/s.
#include "block.hpp"
#include "elem.hpp"
#include "philox.hpp"

namespace rl {

namespace {

template <class T>
__global__ void __launch_bounds__(256) drop_kernel(const typename T::raw* x, typename T::raw* out,
                                                   int64_t count, DropRule rule, bool past) {
  constexpr int V = 16 / T::kBytes;
  const uint64_t seed = rule.seed_at ? *rule.seed_at : rule.seed;
  const int64_t blocks = (count + 7) / 8;
  for (int64_t b = (int64_t)blockIdx.x * 256 + threadIdx.x; b < blocks; b += (int64_t)gridDim.x * 256) {
    const bool whole = 8 * b + 8 <= count;
    Pack<T, V> v[8 / V];
    if (whole) {
#pragma unroll
      for (int i = 0; i < 8 / V; ++i) v[i] = load_pack<T, V>(x + 8 * b + V * i);
    }
    const uint4 d = drop_draws(rule, seed, (uint64_t)b);
    if (whole) {
#pragma unroll
      for (int i = 0; i < 8 / V; ++i) {
#pragma unroll
        for (int j = 0; j < V; ++j)
          v[i].v[j] = draw_of(d, V * i + j) >= rule.drop ? T::narrow(T::widen(v[i].v[j]) * rule.scale)
                                                         : (typename T::raw)0;
        store_pack<T, V>(out + 8 * b + V * i, v[i], past);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t e = 8 * b + j;
        if (e >= count) continue;
        out[e] = draw_of(d, j) >= rule.drop ? T::narrow(T::widen(x[e]) * rule.scale) : (typename T::raw)0;
      }
    }
  }
}

}  // namespace

hipError_t drop_forward_launch(int32_t dtype, const void* x, int64_t count, float p, uint64_t seed,
                               const uint64_t* seed_at, uint32_t offset, void* out, hipStream_t stream) {
  const DropRule rule = drop_rule(p, seed, seed_at, offset);
  const int64_t blocks = (count + 7) / 8, groups = (blocks + 255) / 256;
  const dim3 grid((uint32_t)(groups < (1 << 22) ? groups : 1 << 22));
  const auto run = [&](auto type) {
    using T = decltype(type);
    using raw = typename T::raw;
    drop_kernel<T><<<grid, 256, 0, stream>>>(static_cast<const raw*>(x), static_cast<raw*>(out), count, rule,
                                             count * T::kBytes > kPastBytes);
  };
  if (dtype == POLICY_F32)
    run(F32());
  else if (dtype == POLICY_BF16)
    run(BF16());
  else
    run(F16());
  return hipGetLastError();
}

}  // namespace rl
