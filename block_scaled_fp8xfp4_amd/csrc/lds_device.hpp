// LDS by address, unaligned vectors and waits of the kernels that stage tiles
// through LDS themselves.
#pragma once
#include "mx_device.hpp"

namespace mx {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));
typedef uint32_t u32x2_a1 __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32x4_a1 __attribute__((ext_vector_type(4), aligned(1)));

template <typename V> __device__ __forceinline__ V lds_read(uint32_t addr) {
  return *reinterpret_cast<const __attribute__((address_space(3))) V*>(addr);
}
template <typename V> __device__ __forceinline__ void lds_write(uint32_t addr, const V& v) {
  *reinterpret_cast<__attribute__((address_space(3))) V*>(addr) = v;
}

template <int V> struct Int { static constexpr int value = V; };
template <int N> __device__ __forceinline__ void wait_vm() { asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory"); }

// v, of which the compiler knows nothing: what is made from it inside a loop is not kept in registers outside of it.
__device__ __forceinline__ int fresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

constexpr int XCDS = 8;

}  // namespace mx
