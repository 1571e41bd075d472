// Casts to E4M3 codes with an fp32 scale for each block of 128: along a row
// (activations), of 128 x 128 (weights), along a column (sums over tokens,
// transposed), and of SwiGLU between an FFN's products.
//   scale = max(amax, 2^-60) / 448 (fp32 division), code = the E4M3 value nearest to x / scale, ties to even
// A block that holds an infinity or a NaN has the scale NaN, so every sum over
// it is NaN too.
#include "any_device.hpp"
#include "b128_launch.hpp"
#include "group_device.hpp"

namespace mx {

constexpr uint32_t AMAX_FLOOR = 0x21800000u;      // 2^-60
constexpr uint32_t INF_BITS = 0x7F800000u;

struct Scale128 { float sc, inv; };
// From the bits of a block's largest |x| (as whole numbers magnitudes are in order, infinities and NaN last).
__device__ __forceinline__ Scale128 scale128(uint32_t amax) {
  if (amax >= INF_BITS) return Scale128{__uint_as_float(0x7FC00000u), 0.0f};
  const float sc = __uint_as_float(max(amax, AMAX_FLOOR)) / 448.0f;
  return Scale128{sc, 1.0f / sc};
}

__device__ __forceinline__ uint32_t bits_max(uint32_t m, float x) { return max(m, __float_as_uint(x) & 0x7FFFFFFFu); }

// A number that rounds to the code of x / sc: the product with the reciprocal, which is within 2^-23 of the quotient,
// rounded to 16 bits, and moved by one of its last bits toward the side that the remainder says the quotient is on.  Borders
// between codes have few bits, so the quotient is on the same side of every one of them; it is on one where the remainder is
// zero.  With sc >= 2^-69 no remainder that counts falls under fp32's smallest numbers.  Codes from the product alone, with a
// check for borders nearby, are slower: rows in bf16 meet borders in most wavefronts, since both x and the scale come from 8
// bits (8192 x 4096 27.5 us).
__device__ __forceinline__ float quotient_side(float x, const Scale128& s) {
  const float a = __builtin_fabsf(x);
  const uint32_t b = (__float_as_uint(a * s.inv) + 0x80u) & 0xFFFFFF00u;
  const int r = __float_as_int(__builtin_fmaf(-__uint_as_float(b), s.sc, a));      // an exact zero is +0
  const float q = __uint_as_float(b + (uint32_t)min(max(r, -1), 1));
  return __builtin_copysignf(fminf(q, 448.0f), x);
}

__device__ __forceinline__ uint32_t code_quad(const float* v, const Scale128& s) {
  const int d = __builtin_amdgcn_cvt_pk_fp8_f32(quotient_side(v[0], s), quotient_side(v[1], s), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(quotient_side(v[2], s), quotient_side(v[3], s), d, true);
}
__device__ __forceinline__ u32x2 codes8(const float* v, const Scale128& s) { return u32x2{code_quad(v, s), code_quad(v + 4, s)}; }

// Maximum over the 16 lanes of a DPP row.
__device__ __forceinline__ uint32_t row16_max_bits(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, false));
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, false));
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x124, 0xF, 0xF, false));
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x128, 0xF, 0xF, false));
  return m;
}

// Rows: 16 lanes hold a block, eight columns each; those past the row's end hold zeros and write nothing.
template <bool BF16>
__global__ __launch_bounds__(256) void quantize128_rows_kernel(const void* __restrict__ src, int64_t ld, uint32_t n, uint32_t cols,
                                                               uint32_t nb, uint8_t* __restrict__ q, float* __restrict__ sc) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= n) return;                                                 // whole blocks are in or out
  const uint32_t r = i / (nb * 16), c = (i - r * nb * 16) * 8;
  const bool in = c < cols;
  float v[8] = {};
  if (in) load8(src, BF16, (int64_t)r * ld + c, v);
  uint32_t amax = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = bits_max(amax, v[e]);
  const Scale128 s = scale128(row16_max_bits(amax));
  if (in) *reinterpret_cast<u32x2*>(q + (int64_t)r * cols + c) = codes8(v, s);
  if ((i & 15) == 0) sc[i >> 4] = s.sc;
}

__device__ __forceinline__ float element(const void* p, bool bf16, int64_t i) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16) : static_cast<const float*>(p)[i];
}

// SwiGLU without double arithmetic where the result cannot depend on it.  Near values (fp32) are within 2^-20 of the values
// that the cast is defined on, so a block's largest value is one of those whose near value is within 2^-19 of the largest
// near one: where that is one value, its evaluation in double gives the scale.  A code is that of a near value times the
// reciprocal of the scale if it does not change within NEAR_EPS of it (2^-20 and the roundings of the reciprocal and the
// product); about one wavefront in 60 holds a code that does, and evaluates it in double.  Blocks with several such largest
// values, or out of the range in which near values are good, take the double form as a whole.
//
// What bounds it is instructions (8192 x 4096 bf16 42 to 47 us, 4.0 to 3.6 TB/s; the loads and stores alone 37) and, for few rows, the
// longest way through them (48 x 2048 3.3 us): the largest value is found with its place in its three lowest bits (2^-20
// of it at most) and read again; a near value never reaches past 464, where a code would not be 448, so none is clamped;
// and codes are mended one by one (whole blocks in double instead: 48 x 2048 4.3 us, 999 x 1376 fp32 6.9 from 5.9).  Several
// blocks a lane, whose largest are evaluated at once, cost more registers than they save (8192 x 4096 46 us, 999 x 1376 6.7).
constexpr float NEAR_EPS = 1.25f * 9.5367431640625e-07f;
__device__ __forceinline__ u32x2 codes8_times(const float* v, float f) {
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * f, v[1] * f, 0, false), hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * f, v[5] * f, 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * f, v[3] * f, lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * f, v[7] * f, hi, true);
  return u32x2{(uint32_t)lo, (uint32_t)hi};
}

template <bool BF16>
__global__ __launch_bounds__(256) void swiglu_quantize128_kernel(const void* __restrict__ src, int64_t ld, uint32_t n, uint32_t cols,
                                                                 uint32_t nb, uint8_t* __restrict__ q, float* __restrict__ sc) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= n) return;                                                 // whole blocks are in or out
  const int lane = threadIdx.x & 63, l = lane & 15;
  const uint32_t r = i / (nb * 16), c = (i - r * nb * 16) * 8;
  const bool in = c < cols;
  const int64_t row = (int64_t)r * ld, at = row + c;
  float a[8], gmin = 0.0f;
  uint32_t first = 0, second = 0;                                     // the two largest, with their places
  {
    float g[8] = {}, u[8] = {};
    if (in) {
      load8(src, BF16, at, g);
      load8(src, BF16, at + cols, u);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a[e] = swiglu_near(g[e], u[e]);
      gmin = fminf(gmin, g[e]);
      const uint32_t key = (__float_as_uint(a[e]) & 0x7FFFFFF8u) | (uint32_t)e;                  // NaN is the largest
      second = max(second, min(first, key));
      first = max(first, key);
    }
  }
  const uint32_t top = row16_max_bits(first);
  const float most = __uint_as_float(top & ~7u);
  const uint32_t edge = __float_as_uint(most * (1.0f - 3.814697265625e-06f));                    // 2^-18: 2^-19 and the places
  const uint32_t holds = (uint32_t)(__ballot(first >= edge) >> (lane & 48)) & 0xFFFFu;           // the block's lanes that do
  const bool sure = gmin > SWIGLU_MIN_G && most >= 3.5e-18f && most <= 1.3e36f &&                // 2^-58, 2^120
                    second < edge && (holds & (holds - 1)) == 0;
  const uint32_t place = min(c - l * 8 + __builtin_ctz(holds | 0x8000u) * 8 + (top & 7u), cols - 1);
  const float exact = swiglu(element(src, BF16, row + place), element(src, BF16, row + cols + place));
  Scale128 s = scale128(__float_as_uint(exact) & 0x7FFFFFFFu);
  u32x2 d = codes8_times(a, s.inv * (1.0f - NEAR_EPS));
  const u32x2 hi = codes8_times(a, s.inv * (1.0f + NEAR_EPS));
  if (!__all(sure)) {
    float v[8] = {}, u[8];
    if (in) {                                                         // again, so that they need no registers until then
      load8(src, BF16, at, v);
      load8(src, BF16, at + cols, u);
    }
    uint32_t amax = 0;
#pragma unroll 1
    for (int h = 0; h < 2; ++h)                                       // four at a time: the double form is long
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e / 4 == h) v[e] = in ? swiglu(v[e], u[e]) : 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = bits_max(amax, v[e]);
    s = scale128(row16_max_bits(amax));
    d = codes8(v, s);
  } else if (__any(d[0] != hi[0] || d[1] != hi[1])) {
    uint64_t codes = (uint64_t)d[1] << 32 | d[0];
    const uint64_t open = codes ^ ((uint64_t)hi[1] << 32 | hi[0]);
#pragma unroll 1
    for (int e = 0; e < 8; ++e) {
      const bool ask = (open >> (8 * e) & 0xFF) != 0;                 // never a lane past the row's end: its values are zeros
      if (!__any(ask)) continue;
      const float v = ask ? swiglu(element(src, BF16, at + e), element(src, BF16, at + cols + e)) : 0.0f;
      const uint64_t code = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(quotient_side(v, s), 0.0f, 0, false) & 0xFFu;
      if (ask) codes = (codes & ~(uint64_t(0xFF) << (8 * e))) | code << (8 * e);
    }
    d = u32x2{(uint32_t)codes, (uint32_t)(codes >> 32)};
  }
  if (in) *reinterpret_cast<u32x2*>(q + (int64_t)r * cols + c) = d;
  if (l == 0) sc[i >> 4] = s.sc;
}

hipError_t launch_quantize128_rows(const void* src, bool bf16, int64_t ld, int64_t rows, int64_t cols, bool swiglu,
                                   uint8_t* q, float* sc, hipStream_t stream) {
  const int64_t nb = (cols + 127) / 128, n = rows * nb * 16;
  if (n == 0) return hipSuccess;
  const dim3 grid((unsigned)((n + 255) / 256)), block(256);
#define MX_Q(KERNEL) hipLaunchKernelGGL((KERNEL), grid, block, 0, stream, src, ld, (uint32_t)n, (uint32_t)cols, (uint32_t)nb, q, sc)
  if (bf16) { if (swiglu) MX_Q(swiglu_quantize128_kernel<true>); else MX_Q(quantize128_rows_kernel<true>); }
  else { if (swiglu) MX_Q(swiglu_quantize128_kernel<false>); else MX_Q(quantize128_rows_kernel<false>); }
#undef MX_Q
  return hipGetLastError();
}

// 128 x 128 blocks, a workgroup each: 16 lanes per row, every 16th row.
template <bool BF16>
__global__ __launch_bounds__(256) void quantize128_tiles_kernel(const void* __restrict__ src, int64_t ld, int64_t rows, int64_t cols,
                                                                uint32_t nbr, uint32_t nbc, uint8_t* __restrict__ q,
                                                                float* __restrict__ sc) {
  __shared__ uint32_t part[4];
  const uint32_t per = nbr * nbc, mat = blockIdx.x / per, in = blockIdx.x - mat * per, br = in / nbc, bc = in - br * nbc;
  const int64_t c = (int64_t)bc * 128 + (threadIdx.x & 15) * 8, r0 = (int64_t)br * 128 + (threadIdx.x >> 4);
  const int64_t m0 = (int64_t)mat * rows;                             // matrices follow one another
  float v[8][8];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (c >= cols || r0 + i * 16 >= rows) continue;
    load8(src, BF16, (m0 + r0 + i * 16) * ld + c, v[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = bits_max(amax, v[i][e]);
  }
#pragma unroll
  for (int d = 32; d >= 1; d /= 2) amax = max(amax, (uint32_t)__shfl_xor((int)amax, d));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = amax;
  __syncthreads();
  const Scale128 s = scale128(max(max(part[0], part[1]), max(part[2], part[3])));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (c >= cols || r0 + i * 16 >= rows) continue;
    *reinterpret_cast<u32x2*>(q + (m0 + r0 + i * 16) * cols + c) = codes8(v[i], s);
  }
  if (threadIdx.x == 0) sc[blockIdx.x] = s.sc;
}

hipError_t launch_quantize128_tiles(const void* src, bool bf16, int64_t ld, int64_t count, int64_t rows, int64_t cols,
                                    uint8_t* q, float* sc, hipStream_t stream) {
  const int64_t nbr = (rows + 127) / 128, nbc = (cols + 127) / 128, n = count * nbr * nbc;
  if (n == 0) return hipSuccess;
  const dim3 grid((unsigned)n), block(256);
  if (bf16) hipLaunchKernelGGL(quantize128_tiles_kernel<true>, grid, block, 0, stream, src, ld, rows, cols, (uint32_t)nbr, (uint32_t)nbc, q, sc);
  else hipLaunchKernelGGL(quantize128_tiles_kernel<false>, grid, block, 0, stream, src, ld, rows, cols, (uint32_t)nbr, (uint32_t)nbc, q, sc);
  return hipGetLastError();
}

// Columns: a workgroup takes 128 rows of one group and 64 columns at a time.  A thread holds four rows of eight columns; the columns'
// largest values meet in LDS, where 64 threads make the scales; then each thread's codes go to LDS as dwords of four rows,
// and come out as whole columns of 128 bytes.  A group's rows past its last are zeros.
constexpr int TCOLS = 64;
template <bool BF16>
__global__ __launch_bounds__(256) void quantize128_t_kernel(const void* __restrict__ src, int64_t ld, int64_t rows, int cols,
                                                            const int32_t* __restrict__ offsets, int E, uint8_t* __restrict__ q,
                                                            float* __restrict__ sc, int64_t q_ld, uint32_t ncg, int per) {
  constexpr int PITCH = 33;                                           // dwords per column: 8 columns' writes meet on no bank twice
  __shared__ __attribute__((aligned(16))) uint32_t part[16][TCOLS];
  __shared__ __attribute__((aligned(16))) float scale[TCOLS], inv[TCOLS];
  __shared__ uint32_t code[TCOLS * PITCH];
  const uint32_t b = blockIdx.x / ncg, cg = blockIdx.x - b * ncg;
  int64_t r0 = (int64_t)b * 128, n = rows - r0;
  if (offsets) {
    const GroupTile g = find_tile(offsets, E, rows, 128, b);
    if (g.e < 0) return;
    r0 = g.row0 + (int64_t)g.tile * 128;
    n = g.rows - g.tile * 128;
  }
  n = min(n, (int64_t)128);
  const int c = (threadIdx.x & 7) * 8, rq = threadIdx.x >> 3;         // columns c .. c + 7, rows 4 rq .. 4 rq + 3
  for (int t = 0; t < per; ++t) {
    const int c0 = (int)(cg * per + t) * TCOLS;
    if (c0 >= cols) break;
    float v[4][8];
    uint32_t amax[8] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = (r0 + rq * 4 + i) * ld + c0 + c;
      if (rq * 4 + i >= n) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
      } else if (c0 + c + 8 <= cols) {
        load_any<8>(src, BF16, at, v[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = c0 + c + e < cols ? element(src, BF16, at + e) : 0.0f;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int i = 0; i < 4; ++i) amax[e] = bits_max(amax[e], v[i][e]);
      amax[e] = max(amax[e], (uint32_t)__builtin_amdgcn_mov_dpp((int)amax[e], 0x128, 0xF, 0xF, false));   // the row's other half
    }
    if ((threadIdx.x & 8) == 0) {
      u32x4* const to = reinterpret_cast<u32x4*>(&part[threadIdx.x >> 4][c]);
      to[0] = u32x4{amax[0], amax[1], amax[2], amax[3]};
      to[1] = u32x4{amax[4], amax[5], amax[6], amax[7]};
    }
    __syncthreads();
    if (threadIdx.x < TCOLS) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) m = max(m, part[i][threadIdx.x]);
      const Scale128 s = scale128(m);
      scale[threadIdx.x] = s.sc;
      inv[threadIdx.x] = s.inv;
      if (c0 + (int)threadIdx.x < cols) sc[(int64_t)(c0 + threadIdx.x) * (q_ld / 128) + b] = s.sc;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float col4[4] = {v[0][e], v[1][e], v[2][e], v[3][e]};
      code[(c + e) * PITCH + rq] = code_quad(col4, Scale128{scale[c + e], inv[c + e]});
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 2; ++p) {                                       // eight lanes write a column
      const int col = p * 32 + rq, k = (threadIdx.x & 7) * 4;
      if (c0 + col >= cols) continue;
      const uint32_t* const from = &code[col * PITCH + k];
      *reinterpret_cast<u32x4*>(q + (int64_t)(c0 + col) * q_ld + (int64_t)b * 128 + k * 4) = u32x4{from[0], from[1], from[2], from[3]};
    }
  }
}

hipError_t launch_quantize128_t(const void* src, bool bf16, int64_t ld, int64_t rows, int cols, const int32_t* offsets,
                                int E, uint8_t* q, float* sc, int64_t q_ld, hipStream_t stream) {
  const int64_t nb = offsets ? q_ld / 128 : (rows + 127) / 128, nct = (cols + TCOLS - 1) / TCOLS;
  // a workgroup finds its group once for two column tiles where there are many (bf16 from memory in 64 groups: 32768 x 2048 55
  // us, for one 60, 4096 x 4096 30.2 and 31.9; with fewer tiles 4096 x 2048 18.4 and 18.7, 16384 x 1024 22.5 and 21.9)
  const int per = nb * nct > 4096 ? 2 : 1;
  const int64_t ncg = (nct + per - 1) / per;
  if (nb * ncg == 0) return hipSuccess;
  const dim3 grid((unsigned)(nb * ncg)), block(256);
  if (bf16) hipLaunchKernelGGL(quantize128_t_kernel<true>, grid, block, 0, stream, src, ld, rows, cols, offsets, E, q, sc, q_ld, (uint32_t)ncg, per);
  else hipLaunchKernelGGL(quantize128_t_kernel<false>, grid, block, 0, stream, src, ld, rows, cols, offsets, E, q, sc, q_ld, (uint32_t)ncg, per);
  return hipGetLastError();
}

}  // namespace mx
