// Block-32 quantizer kernel: fp32 or bf16 rows -> E4M3 bytes or packed E2M1
// nibbles plus one E8M0 scale per 32 values (the per-block FP8/FP4 casts of
// the "New Deepseek 4.1 flash recipe" thread, post #6, "Why TileLang"; the
// conversion rule is OCP MX v1.0's).  One thread per block of 32: a thread
// reads 64-128 contiguous bytes and its neighbours the next ones, so a wave
// streams a contiguous span of the row-major source.
#include "mx_cast.hpp"
#include "mx_launch.hpp"

namespace mx {

template <bool BF16, bool FP4>
__global__ __launch_bounds__(256) void quantize_kernel(const void* __restrict__ src, int64_t nblocks,
                                                       uint8_t* __restrict__ q, uint8_t* __restrict__ sc) {
  const int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= nblocks) return;
  float v[32];
  if (BF16) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(src) + b * 32);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x4 d = p[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[8 * i + 2 * j] = __uint_as_float(d[j] << 16);
        v[8 * i + 2 * j + 1] = __uint_as_float(d[j] & 0xFFFF0000u);
      }
    }
  } else {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const float*>(src) + b * 32);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const u32x4 d = p[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] = __uint_as_float(d[j]);
    }
  }
  if (FP4) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) amax = fmaxf(amax, __builtin_fabsf(v[i]));
    const uint32_t s = e8m0_code_for_amax(amax, 2);
    u32x4 out;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t d = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) d |= encode_e2m1(v[8 * w + i], s) << (4 * i);
      out[w] = d;
    }
    *reinterpret_cast<u32x4*>(q + b * 16) = out;
    sc[b] = (uint8_t)s;
  } else {
    uint32_t out[8];
    const uint32_t s = quantize32_e4m3(v, out);
    u32x4* dst = reinterpret_cast<u32x4*>(q + b * 32);
    dst[0] = u32x4{out[0], out[1], out[2], out[3]};
    dst[1] = u32x4{out[4], out[5], out[6], out[7]};
    sc[b] = (uint8_t)s;
  }
}

hipError_t launch_quantize(const void* src, bool bf16, int64_t rows, int64_t cols, bool fp4,
                           uint8_t* q, uint8_t* sc, hipStream_t stream) {
  const int64_t nblocks = rows * (cols / 32);
  if (nblocks == 0) return hipSuccess;
  const dim3 block(256), grid((unsigned)((nblocks + 255) / 256));
  if (bf16 && fp4) hipLaunchKernelGGL((quantize_kernel<true, true>), grid, block, 0, stream, src, nblocks, q, sc);
  else if (bf16) hipLaunchKernelGGL((quantize_kernel<true, false>), grid, block, 0, stream, src, nblocks, q, sc);
  else if (fp4) hipLaunchKernelGGL((quantize_kernel<false, true>), grid, block, 0, stream, src, nblocks, q, sc);
  else hipLaunchKernelGGL((quantize_kernel<false, false>), grid, block, 0, stream, src, nblocks, q, sc);
  return hipGetLastError();
}

// Codes and scales back to the values they stand for (exact in fp32; bf16
// holds every element times its scale too, except where the product falls
// under bf16's smallest values, rounded to nearest even there): the inverse
// of the casts above, for a caller's own operations on quantized rows.  One
// thread per 8 elements, so a wave reads 256 or 512 contiguous bytes and
// writes 1 or 2 KB: memory-bound (8192 x 4096 E2M1 to bf16 17.8 us, 4.7 TB/s).
template <bool FP4>
__global__ __launch_bounds__(256) void dequantize_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ sc,
                                                         int64_t nchunks, void* __restrict__ out, bool bf16) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= nchunks) return;
  const int e = (int)sc[c >> 2] - 127;
  float v[8];
  if (FP4) {
    const uint32_t d = *reinterpret_cast<const uint32_t*>(q + c * 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t code = (d >> (4 * j)) & 15u, m = code & 7u;
      const uint32_t mag = m == 0 ? 0u : (m == 1 ? 0x3F000000u : (((m >> 1) + 126u) << 23) | ((m & 1u) << 22));
      v[j] = __builtin_ldexpf(__uint_as_float(mag | ((code & 8u) << 28)), e);
    }
  } else {
    const uint2 d = *reinterpret_cast<const uint2*>(q + c * 8);
    v[0] = __builtin_amdgcn_cvt_f32_fp8(d.x, 0); v[1] = __builtin_amdgcn_cvt_f32_fp8(d.x, 1);
    v[2] = __builtin_amdgcn_cvt_f32_fp8(d.x, 2); v[3] = __builtin_amdgcn_cvt_f32_fp8(d.x, 3);
    v[4] = __builtin_amdgcn_cvt_f32_fp8(d.y, 0); v[5] = __builtin_amdgcn_cvt_f32_fp8(d.y, 1);
    v[6] = __builtin_amdgcn_cvt_f32_fp8(d.y, 2); v[7] = __builtin_amdgcn_cvt_f32_fp8(d.y, 3);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __builtin_ldexpf(v[j], e);
  }
  store8(out, bf16, c * 8, v);
}

hipError_t launch_dequantize(const uint8_t* q, const uint8_t* sc, bool fp4, int64_t rows, int64_t cols, void* out,
                             bool bf16, hipStream_t stream) {
  const int64_t n = rows * (cols / 8);
  if (n == 0) return hipSuccess;
  const dim3 grid((unsigned)((n + 255) / 256)), block(256);
  if (fp4) hipLaunchKernelGGL(dequantize_kernel<true>, grid, block, 0, stream, q, sc, n, out, bf16);
  else hipLaunchKernelGGL(dequantize_kernel<false>, grid, block, 0, stream, q, sc, n, out, bf16);
  return hipGetLastError();
}

// SwiGLU + block-32 codes of gate/up rows [T][2I] (gate, then up): what lies
// between the two products of an FFN.  a = silu(gate) * up in double, rounded
// once to fp32 (swiglu, as in every other kernel of the library), then the
// block's codes: from fp32 values where those decide the codes (codes_near),
// in double for the wavefronts that hold one that they do not.  One thread per
// 8 columns of one row.
template <bool BF16, bool FP4>
__global__ __launch_bounds__(256) void swiglu_quantize_kernel(const void* __restrict__ gu, int64_t ld, int64_t nchunks,
                                                              int I, uint8_t* __restrict__ q, uint8_t* __restrict__ sc) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= nchunks) return;                                     // whole quads are in or out (I % 32 == 0)
  const int per_row = I / 8;
  const int64_t t = c / per_row, i = (c - t * per_row) * 8;
  float g[8], u[8];
  load8(gu, BF16, t * ld + i, g);
  load8(gu, BF16, t * ld + I + i, u);
  uint32_t d[2];
  const uint32_t s = swiglu_codes8<FP4>(g, u, d);
  if (FP4) *reinterpret_cast<uint32_t*>(q + c * 4) = d[0];
  else *reinterpret_cast<uint2*>(q + c * 8) = uint2{d[0], d[1]};
  if ((c & 3) == 0) sc[c >> 2] = (uint8_t)s;
}

hipError_t launch_swiglu_quantize(const void* gu, bool bf16, int64_t ld, int64_t T, int I, bool fp4, uint8_t* q,
                                  uint8_t* sc, hipStream_t stream) {
  const int64_t n = T * (I / 8);
  if (n == 0) return hipSuccess;
  const dim3 grid((unsigned)((n + 255) / 256)), block(256);
#define MX_SQ(B, F) hipLaunchKernelGGL((swiglu_quantize_kernel<B, F>), grid, block, 0, stream, gu, ld, n, I, q, sc)
  if (bf16) { if (fp4) MX_SQ(true, true); else MX_SQ(true, false); }
  else { if (fp4) MX_SQ(false, true); else MX_SQ(false, false); }
#undef MX_SQ
  return hipGetLastError();
}

// Diagnostic: the finite floats whose magnitude bits lie in [lo, hi), with
// both signs, through both E4M3 encoders of the intermediate: the hardware
// conversion of requant2_e4m3 and the integer rounding of encode_e4m3 (scale
// code 127: the value itself is encoded).  Mismatches are added to *nbad.
__global__ __launch_bounds__(256) void check_requant_kernel(uint32_t lo, uint32_t hi, unsigned long long* nbad) {
  unsigned long long bad = 0;
  for (uint64_t i = lo + (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; i < hi; i += (uint64_t)gridDim.x * blockDim.x) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const float v = __uint_as_float((uint32_t)i | (s ? 0x80000000u : 0u));
      bad += (requant2_e4m3(v, 0.0f, 127) & 0xFFu) != encode_e4m3(v, 127);
    }
  }
  if (bad) atomicAdd(nbad, bad);
}

hipError_t launch_check_requant(uint32_t lo, uint32_t hi, unsigned long long* nbad, hipStream_t stream) {
  if (lo >= hi) return hipSuccess;
  hipLaunchKernelGGL(check_requant_kernel, dim3(2048), dim3(256), 0, stream, lo, hi, nbad);
  return hipGetLastError();
}

}  // namespace mx

namespace mx {

// Weight prefetch (spark-ds41f README, "Current baseline": L2 weight prefetch
// during decode, the next layer's weights and scale words streamed in while
// latency-bound kernels run; TP4 README, settings table, row "L2 prefetch": a
// side-stream kernel during idle phases, data untouched).  Workgroup i reads
// chunk i of the range, so the chunk lands in the L2 of the XCD that runs
// workgroup i and in the memory-side cache (MALL) shared by every XCD.  The
// reads are LDS DMA into a scratch row per wavefront (no register ever holds
// them, nothing is kept); the workgroup waits for all of them before it ends.
// Whole 16-byte units only (p 16-byte aligned, chunk a multiple of 16).
__global__ __launch_bounds__(256) void prefetch_kernel(const uint8_t* __restrict__ p, uint64_t bytes, uint64_t chunk) {
  __shared__ u32x4 scratch[256];
  const int wave = threadIdx.x >> 6;
  const uint64_t c0 = (uint64_t)blockIdx.x * chunk;
  const uint64_t c1 = c0 + chunk < bytes ? c0 + chunk : bytes;
  for (uint64_t off = c0 + (uint64_t)threadIdx.x * 16; off + 16 <= c1; off += 256 * 16)
    dma16_to_lds(p + off, &scratch[wave * 64]);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

hipError_t launch_prefetch(const void* p, uint64_t bytes, uint64_t chunk, hipStream_t stream) {
  const uint64_t n = (bytes + chunk - 1) / chunk;
  hipLaunchKernelGGL(prefetch_kernel, dim3((unsigned)n), dim3(256), 0, stream, static_cast<const uint8_t*>(p), bytes,
                     chunk);
  return hipGetLastError();
}

}  // namespace mx
