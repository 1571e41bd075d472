// Elements of rows that start at any place their type allows.
#pragma once
#include "lds_device.hpp"
#include "mx_cast.hpp"

namespace mx {

// N elements from element i on, at any alignment that the type allows.  ONCE: nothing reads them again (FAR: nothing reads
// them soon), so the caches need not keep them.
template <int N, bool ONCE = false> __device__ __forceinline__ void load_any(const void* p, bool bf16, int64_t i, float* v) {
  if (N == 1) {
    v[0] = bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16) : static_cast<const float*>(p)[i];
  } else if (bf16) {
    const u32x4_a1* const s = reinterpret_cast<const u32x4_a1*>(static_cast<const uint16_t*>(p) + i);
    const u32x4 d = ONCE ? __builtin_nontemporal_load(s) : *s;
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      v[2 * j] = __uint_as_float(d[j] << 16);
      v[2 * j + 1] = __uint_as_float(d[j] & 0xFFFF0000u);
    }
  } else {
    const u32x4_a1* s = reinterpret_cast<const u32x4_a1*>(static_cast<const float*>(p) + i);
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
      const u32x4 d = ONCE ? __builtin_nontemporal_load(s + q) : s[q];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * q + j] = __uint_as_float(d[j]);
    }
  }
}
template <int N, bool FAR = false> __device__ __forceinline__ void store_any(void* p, bool bf16, int64_t i, const float* v) {
  if (N == 1) {
    if (bf16) static_cast<uint16_t*>(p)[i] = (uint16_t)bf16_pair(v[0], 0.0f);
    else static_cast<float*>(p)[i] = v[0];
  } else if (bf16) {
    u32x4 d;
#pragma unroll
    for (int j = 0; j < N / 2; ++j) d[j] = bf16_pair(v[2 * j], v[2 * j + 1]);
    u32x4_a1* const to = reinterpret_cast<u32x4_a1*>(static_cast<uint16_t*>(p) + i);
    if constexpr (FAR) __builtin_nontemporal_store(d, to);
    else *to = d;
  } else {
    u32x4_a1* s = reinterpret_cast<u32x4_a1*>(static_cast<float*>(p) + i);
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
      const u32x4 d = {__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                       __float_as_uint(v[4 * q + 3])};
      if constexpr (FAR) __builtin_nontemporal_store(d, s + q);
      else s[q] = d;
    }
  }
}

}  // namespace mx
