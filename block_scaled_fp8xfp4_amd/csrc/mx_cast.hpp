// Device-side building blocks of the dense block's kernels (norm, SwiGLU
// cast, dequantize, FP4 products): rows in chunks of 8 elements per lane,
// block-32 codes by the hardware conversions, SwiGLU + codes.
#pragma once
#include "mx_device.hpp"

namespace mx {

// Two floats -> bf16 in one hardware conversion: the bits of f32_to_bf16_rne
// for every float but NaN (all of them compared).  a in the low half.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// ---------------------------------------------------------------------------
// Rows in chunks of 8 consecutive elements per lane: four neighbouring lanes
// (a quad) hold one block of 32.

// 8 fp32 or bf16 elements from element i on (i % 8 == 0, 16-byte aligned).
__device__ __forceinline__ void load8(const void* p, bool bf16, int64_t i, float* v) {
  if (bf16) {
    const u32x4 d = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(d[j] << 16);
      v[2 * j + 1] = __uint_as_float(d[j] & 0xFFFF0000u);
    }
  } else {
    const u32x4* s = reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + i);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const u32x4 d = s[q];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * q + j] = __uint_as_float(d[j]);
    }
  }
}

__device__ __forceinline__ void store8(void* p, bool bf16, int64_t i, const float* v) {
  if (bf16) {
    u32x4 d;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      d[j] = bf16_pair(v[2 * j], v[2 * j + 1]);
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) = d;
  } else {
    u32x4* d = reinterpret_cast<u32x4*>(static_cast<float*>(p) + i);
#pragma unroll
    for (int q = 0; q < 2; ++q)
      d[q] = u32x4{__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                   __float_as_uint(v[4 * q + 3])};
  }
}

// Maximum over a quad (lanes 4 r .. 4 r + 3), in registers.
__device__ __forceinline__ float quad_max(float m) {
  m = fmaxf(m, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(m), 0xB1, 0xF, 0xF, false)));   // quad [1,0,3,2]
  m = fmaxf(m, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(m), 0x4E, 0xF, 0xF, false)));   // quad [2,3,0,1]
  return m;
}

// Codes of N elements under scale code sc by the hardware conversions (round
// to nearest even; E4M3 clamped to +-448 first, E2M1 saturates at +-6 by
// itself): N / 4 dwords of E4M3 or N / 8 of E2M1.  Bit for bit encode_e4m3
// and encode_e2m1 (every finite float compared).  f: 2^(127 - sc), possibly
// times a number next to 1.
template <bool FP4, int N>
__device__ __forceinline__ void codes_scaled(const float* v, float f, uint32_t* out) {
  if (FP4) {
#pragma unroll
    for (int w = 0; w < N / 8; ++w) {
      uint32_t d = 0;
      d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[8 * w] * f, v[8 * w + 1] * f, 1.0f, 0);
      d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[8 * w + 2] * f, v[8 * w + 3] * f, 1.0f, 1);
      d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[8 * w + 4] * f, v[8 * w + 5] * f, 1.0f, 2);
      d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[8 * w + 6] * f, v[8 * w + 7] * f, 1.0f, 3);
      out[w] = d;
    }
  } else {
    auto cl = [](float t) { return __builtin_amdgcn_fmed3f(t, -448.0f, 448.0f); };
#pragma unroll
    for (int w = 0; w < N / 4; ++w) {
      int d = __builtin_amdgcn_cvt_pk_fp8_f32(cl(v[4 * w] * f), cl(v[4 * w + 1] * f), 0, false);
      out[w] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(cl(v[4 * w + 2] * f), cl(v[4 * w + 3] * f), d, true);
    }
  }
}

// Codes of this lane's chunk of a block-32 row (all four lanes of its quad
// active): chunk number `chunk` of the code array (8 or 4 bytes each), and
// one scale byte per quad.
template <bool FP4>
__device__ __forceinline__ void store8_codes(const float* v, uint8_t* q, uint8_t* sc, int64_t chunk) {
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, __builtin_fabsf(v[j]));
  const uint32_t s = e8m0_code_for_amax(quad_max(amax), FP4 ? 2 : 8);
  uint32_t d[2];
  codes_scaled<FP4, 8>(v, __builtin_ldexpf(1.0f, 127 - (int)s), d);
  if (FP4) *reinterpret_cast<uint32_t*>(q + chunk * 4) = d[0];
  else *reinterpret_cast<uint2*>(q + chunk * 8) = uint2{d[0], d[1]};
  if ((chunk & 3) == 0) sc[chunk >> 2] = (uint8_t)s;
}

// ---------------------------------------------------------------------------
// SwiGLU + codes without double arithmetic where the result cannot depend on
// it.  The codes are defined by swiglu() (double, rounded once to fp32); an
// fp32 value a within SWIGLU_EPS of that determines them too if a (1 - eps)
// and a (1 + eps) have the same codes and the block's largest a has the same
// exponent at both ends.  About one element in 2^15 fails that; then the
// wavefront takes the double form.
//
// Error of swiglu_near for g > -60: the exponent's argument is carried in two
// floats, v_exp_f32 and v_rcp_f32 are within 1 ulp, five more roundings, the
// last two those of the products: under half of 2^-20 while the results of
// both products are normal (worst over every float g, with ups of 1 and at
// random, 2^-21.75).  The sigmoid is multiplied by u first: the
// product is subnormal only where u is under 2^-39 at most, and then either
// the sigmoid is 1 (g > 16.7) and the product exact, or the result is under
// 2^-120, which every block that near_block accepts rounds to zero (its codes'
// smallest border is 2^-118).  g / 2 in place of it would lose bits of a
// subnormal g that a large u brings back.
constexpr float SWIGLU_EPS = 9.5367431640625e-07f;               // 2^-20
constexpr float SWIGLU_MIN_G = -60.0f;                           // below: 1 / (1 + e^-g) loses bits to small numbers

__device__ __forceinline__ float swiglu_near(float g, float u) {
  const float h = g * -1.44269504f;                              // -g log2 e = h + l
  const float l = __builtin_fmaf(g, -1.44269504f, -h) - g * 1.92596303e-8f;
  const float e = __builtin_amdgcn_exp2f(h);
  return g * (__builtin_amdgcn_rcpf(1.0f + __builtin_fmaf(e, l * 0.693147181f, e)) * u);
}

// The larger of m and |a|, NaN if either is one (fmaxf would drop it): a near
// value is NaN where its gate's exponent argument overflows (2.36e38 and up),
// and such a block's codes are the double form's.
__device__ __forceinline__ float near_max(float m, float a) { return __builtin_elementwise_maximum(m, __builtin_fabsf(a)); }

// Whether a block whose largest near value is amax can be cast from near
// values: in a range where fp32 keeps its precision (zero is not), and with
// one exponent at both ends.  False for NaN, which a maximum over lanes may
// drop again: each lane asks for its own near_max too.
__device__ __forceinline__ bool near_block(float amax) {
  return amax >= 7.9e-31f && amax <= 1.3e36f &&                  // 2^-100, 2^120
         ((__float_as_uint(amax * (1.0f - SWIGLU_EPS)) ^ __float_as_uint(amax * (1.0f + SWIGLU_EPS))) >> 23) == 0;
}

// Codes of N near values; false if they depend on what near leaves open.
template <bool FP4, int N>
__device__ __forceinline__ bool codes_near(const float* v, uint32_t sc, uint32_t* out) {
  const float f = __builtin_ldexpf(1.0f, 127 - (int)sc);
  uint32_t other[FP4 ? N / 8 : N / 4], diff = 0;
  codes_scaled<FP4, N>(v, f * (1.0f - SWIGLU_EPS), out);
  codes_scaled<FP4, N>(v, f * (1.0f + SWIGLU_EPS), other);
#pragma unroll
  for (int i = 0; i < (FP4 ? N / 8 : N / 4); ++i) diff |= out[i] ^ other[i];
  return diff == 0;
}

// Codes of silu(g) * u of this lane's 8 columns of a block (a quad of lanes): from fp32 values where those decide them in
// the whole wavefront, else in double.  Returns the block's scale.
template <bool FP4> __device__ __forceinline__ uint32_t swiglu_codes8(const float* g, const float* u, uint32_t* d) {
  float a[8], amax = 0.0f, gmin = g[0];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    a[j] = swiglu_near(g[j], u[j]);
    amax = near_max(amax, a[j]);
    gmin = fminf(gmin, g[j]);
  }
  const bool whole = amax == amax;
  amax = quad_max(amax);
  uint32_t s = e8m0_code_for_amax(amax, FP4 ? 2 : 8);
  const bool sure = whole && gmin > SWIGLU_MIN_G && near_block(amax) && codes_near<FP4, 8>(a, s, d);
  if (!__all(sure)) {
    amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      a[j] = swiglu(g[j], u[j]);
      amax = fmaxf(amax, __builtin_fabsf(a[j]));
    }
    s = e8m0_code_for_amax(quad_max(amax), FP4 ? 2 : 8);
    codes_scaled<FP4, 8>(a, __builtin_ldexpf(1.0f, 127 - (int)s), d);
  }
  return s;
}

}  // namespace mx
