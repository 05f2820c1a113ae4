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
// The address needs an element's alignment only: gfx950 loads and stores
// such accesses whole, and rows of any width and stride then take the same
// path as aligned ones.
template <class T, int V>
struct alignas(T::kBytes) Pack {
  typename T::raw v[V];
};

// 16 bytes in registers, and at an address aligned to a 2-byte element.
typedef uint32_t quad_value __attribute__((ext_vector_type(4)));
typedef uint32_t quad __attribute__((ext_vector_type(4), aligned(2)));

template <class T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const typename T::raw* p) {
  if constexpr (V * T::kBytes == 16) {
    return __builtin_bit_cast(Pack<T, V>, (quad_value)*reinterpret_cast<const quad*>(p));
  } else {
    return *reinterpret_cast<const Pack<T, V>*>(p);
  }
}
template <class T, int V>
__device__ __forceinline__ void store_pack(typename T::raw* p, const Pack<T, V>& x) {
  *reinterpret_cast<Pack<T, V>*>(p) = x;
}
// The same past the caches, for outputs too large to be found there again.
template <class T, int V>
__device__ __forceinline__ void store_pack(typename T::raw* p, const Pack<T, V>& x, bool past) {
  if constexpr (V * T::kBytes == 16) {
    const quad_value q = __builtin_bit_cast(quad_value, x);
    if (past) {
      // (the empty statements keep the compiler from merging the two stores
      // into one, which would drop the hint)
      asm volatile("" ::: "memory");
      __builtin_nontemporal_store((quad)q, reinterpret_cast<quad*>(p));
      asm volatile("" ::: "memory");
    } else {
      *reinterpret_cast<quad*>(p) = q;
    }
  } else {
    store_pack<T, V>(p, x);
  }
}
// Outputs above this many bytes are stored past the caches.  A copy of 256 MiB
// measured 90 us through them and 73 us past them; a smaller output is worth
// more to its reader in the 256 MiB cache than the store saves.
constexpr int64_t kPastBytes = (int64_t)96 << 20;
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

// The same at an address that all lanes share plus an offset of each in bytes:
// one scalar and one 32-bit register, no arithmetic per lane.  (The empty
// statement keeps the compiler from adding the offset first and the step to
// every lane's 64-bit sum instead.)
#define RL_GLOBAL __attribute__((address_space(1)))
typedef quad RL_GLOBAL* global_quad;
__device__ __forceinline__ RL_GLOBAL char* shared_address(const void* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  uint64_t a = (uint64_t)hi << 32 | lo;
  asm("" : "+s"(a));
  return reinterpret_cast<RL_GLOBAL char*>(a);
}
template <class T, int V>
__device__ __forceinline__ Pack<T, V> load_pack_at(const void* base, uint32_t off) {
  RL_GLOBAL char* p = shared_address(base) + off;
  if constexpr (V * T::kBytes == 16) {
    return __builtin_bit_cast(Pack<T, V>, (quad_value)*reinterpret_cast<global_quad>(p));
  } else if constexpr (V * T::kBytes == 8) {
    typedef uint32_t two_value __attribute__((ext_vector_type(2)));
    typedef uint32_t two __attribute__((ext_vector_type(2), aligned(2)));
    return __builtin_bit_cast(Pack<T, V>, (two_value)*reinterpret_cast<two RL_GLOBAL*>(p));
  } else if constexpr (V * T::kBytes == 4) {
    typedef uint32_t one __attribute__((aligned(2)));
    return __builtin_bit_cast(Pack<T, V>, (uint32_t)*reinterpret_cast<one RL_GLOBAL*>(p));
  } else {
    return __builtin_bit_cast(Pack<T, V>, *reinterpret_cast<uint16_t RL_GLOBAL*>(p));
  }
}
template <class T, int V>
__device__ __forceinline__ void store_pack_at(void* base, uint32_t off, const Pack<T, V>& x) {
  RL_GLOBAL char* p = shared_address(base) + off;
  if constexpr (V * T::kBytes == 16) {
    *reinterpret_cast<global_quad>(p) = __builtin_bit_cast(quad_value, x);
  } else if constexpr (V * T::kBytes == 8) {
    typedef uint32_t two_value __attribute__((ext_vector_type(2)));
    typedef uint32_t two __attribute__((ext_vector_type(2), aligned(2)));
    *reinterpret_cast<two RL_GLOBAL*>(p) = __builtin_bit_cast(two_value, x);
  } else if constexpr (V * T::kBytes == 4) {
    typedef uint32_t one __attribute__((aligned(2)));
    *reinterpret_cast<one RL_GLOBAL*>(p) = __builtin_bit_cast(uint32_t, x);
  } else {
    *reinterpret_cast<uint16_t RL_GLOBAL*>(p) = __builtin_bit_cast(uint16_t, x);
  }
}

// Elements e .. e + V - 1 of an array of n >= V: the access is moved back to
// lie inside the array (load_inside), and the elements that exist are put in
// their places when they are used (settle), so that the load sits behind no
// branch.  Lanes with e >= n load the last V and use nothing.
template <class T, int V>
__device__ __forceinline__ Pack<T, V> load_inside(const typename T::raw* p, int32_t e, int32_t n) {
  return load_pack<T, V>(p + min(e, n - V));
}
template <class T, int V>
__device__ __forceinline__ void settle(Pack<T, V>& x, int32_t e, int32_t n) {
  if constexpr (V * T::kBytes == 16) {
    const int32_t back = e - (n - V);
    if (back > 0 && back < V)
      x = __builtin_bit_cast(Pack<T, V>, __builtin_bit_cast(unsigned __int128, x) >> (8 * T::kBytes * back));
  }
}

inline bool aligned_to(const void* p, size_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

}  // namespace rl
