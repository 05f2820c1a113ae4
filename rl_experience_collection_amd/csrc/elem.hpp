// Elements of the policy operators: fp32, bf16 and fp16 values loaded,
// widened to fp32, rounded once (nearest even) and stored, a few at a time.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rl {

struct F32 {
  using raw = uint32_t;
  static constexpr int kBytes = 4;
  static __device__ __forceinline__ float widen(raw r) { return __uint_as_float(r); }
  static __device__ __forceinline__ raw narrow(float x) { return __float_as_uint(x); }
};
struct BF16 {
  using raw = uint16_t;
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ float widen(raw r) { return __uint_as_float((uint32_t)r << 16); }
  static __device__ __forceinline__ raw narrow(float x) {
    return __builtin_bit_cast(uint16_t, (__bf16)x);
  }
};
struct F16 {
  using raw = uint16_t;
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ float widen(raw r) {
    return (float)__builtin_bit_cast(_Float16, r);
  }
  static __device__ __forceinline__ raw narrow(float x) {
    return __builtin_bit_cast(uint16_t, (_Float16)x);
  }
};

// V consecutive elements as one memory access (V * kBytes of 2, 4, 8 or 16).
template <class T, int V>
struct alignas(V * T::kBytes) Pack {
  typename T::raw v[V];
};

template <class T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const typename T::raw* p) {
  return *reinterpret_cast<const Pack<T, V>*>(p);
}
template <class T, int V>
__device__ __forceinline__ void store_pack(typename T::raw* p, const Pack<T, V>& x) {
  *reinterpret_cast<Pack<T, V>*>(p) = x;
}
template <class T, int V>
__device__ __forceinline__ void widen_pack(const Pack<T, V>& x, float (&f)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = T::widen(x.v[i]);
}
template <class T, int V>
__device__ __forceinline__ Pack<T, V> narrow_pack(const float (&f)[V]) {
  Pack<T, V> x;
#pragma unroll
  for (int i = 0; i < V; ++i) x.v[i] = T::narrow(f[i]);
  return x;
}

inline bool aligned_to(const void* p, size_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

}  // namespace rl
