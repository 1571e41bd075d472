// Dense products with MXFP4 weights: y[M][N] = a[M][K] . w[N][K]^T, E2M1
// weights and E4M3 or E2M1 activations, both with block-32 E8M0 scales
// ("New Deepseek 4.1 flash recipe" thread, post #6, "How it works":
// block-scaled MMAs, FP8 x FP4; the checkpoint's weights are FP4), and the
// dense SwiGLU FFN made of two of them.
//
// Canonical order: one MFMA chain per output element over all K in order,
// started from zero.  The matrix cores take K in pieces of 64 inside either
// shape: one 16x16x128 step gives, bit for bit, what two chained 32x32x64
// steps give (measured on MI355X for both activation formats, with scales up
// to 2^24 apart), so the kernels below use the shape that suits them and a
// row's result does not depend on M or on the kernel.
#include "mx_device.hpp"
#include "mx_launch.hpp"

namespace mx {

// E2M1 (A) x E2M1 (B) step, K = 128.
__device__ __forceinline__ v4f mfma_fp4_fp4(const v8i& a, const v8i& b, v4f c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// Few rows: one wavefront per 16 columns and 16 rows, operands straight to
// registers.  Lane l serves row / column l % 16; lanes past M or N repeat the
// last row / column, their results are not stored.  K past the end is zero
// elements under scale 1.
template <bool FP4A>
__global__ __launch_bounds__(256) void fp4_rows_kernel(const uint8_t* __restrict__ a, const uint8_t* __restrict__ a_sc,
                                                       const uint8_t* __restrict__ w, const uint8_t* __restrict__ w_sc,
                                                       int M, int N, int K, void* __restrict__ y, bool bf16_out) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = lane & 15, g = lane >> 4;
  const int64_t n0 = ((int64_t)blockIdx.x * 4 + wave) * 16;
  const int64_t m0 = (int64_t)blockIdx.y * 16;
  if (n0 >= N) return;
  const int64_t n = n0 + col < N ? n0 + col : N - 1, m = m0 + col < M ? m0 + col : M - 1;
  const int nblk = K / 32;
  const uint8_t* wp = w + n * (K / 2);
  const uint8_t* wsp = w_sc + n * nblk;
  const uint8_t* ap = a + m * (FP4A ? K / 2 : K);
  const uint8_t* asp = a_sc + m * nblk;
  v4f acc = {0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < K; k += KSTEP) {
    v8i av = {0, 0, 0, 0, 0, 0, 0, 0}, bv = {0, 0, 0, 0, 0, 0, 0, 0};
    uint32_t sa = 127, sb = 127;
    const int blk = k / 32 + g;
    if (blk < nblk) {
      const u32x4 d = ldg16(wp + blk * 16);
      bv = v8i{(int)d[0], (int)d[1], (int)d[2], (int)d[3], 0, 0, 0, 0};
      sb = wsp[blk];
      sa = asp[blk];
      if (FP4A) {
        const u32x4 e = ldg16(ap + blk * 16);
        av = v8i{(int)e[0], (int)e[1], (int)e[2], (int)e[3], 0, 0, 0, 0};
      }
    }
    if (!FP4A) {
      u32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
      if (k + 16 * g < K) lo = ldg16(ap + k + 16 * g);
      if (k + 64 + 16 * g < K) hi = ldg16(ap + k + 64 + 16 * g);
      av = v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
    }
    acc = FP4A ? mfma_fp4_fp4(av, bv, acc, sa, sb) : mfma_fp8_fp4(av, bv, acc, sa, sb);
  }
  if (n0 + col < N)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = m0 + 4 * g + i;
      if (r < M) {
        if (bf16_out) static_cast<uint16_t*>(y)[r * N + n] = f32_to_bf16_rne(acc[i]);
        else static_cast<float*>(y)[r * N + n] = acc[i];
      }
    }
}

hipError_t launch_fp4_gemm(const uint8_t* a, const uint8_t* a_sc, bool fp4a, const uint8_t* w, const uint8_t* w_sc,
                           int M, int N, int K, void* y, bool bf16_out, hipStream_t stream, const char** variant) {
  const dim3 grid((unsigned)((N + 63) / 64), (unsigned)((M + 15) / 16)), block(256);
  if (fp4a) hipLaunchKernelGGL(fp4_rows_kernel<true>, grid, block, 0, stream, a, a_sc, w, w_sc, M, N, K, y, bf16_out);
  else hipLaunchKernelGGL(fp4_rows_kernel<false>, grid, block, 0, stream, a, a_sc, w, w_sc, M, N, K, y, bf16_out);
  *variant = fp4a ? "fp4:rows16_a4" : "fp4:rows16_a8";
  return hipGetLastError();
}

static size_t a256(size_t b) { return (b + 255) / 256 * 256; }

// [gate/up T x 2I fp32][codes of the intermediate][its scales]
size_t fp4_ffn_ws_bytes(int T, int H, int I, bool fp4mid) {
  (void)H;
  return a256((size_t)T * 2 * I * 4) + a256((size_t)T * (fp4mid ? I / 2 : I)) + a256((size_t)T * (I / 32));
}

hipError_t launch_fp4_ffn(const uint8_t* x, const uint8_t* x_sc, bool fp4x, int T, int H, const uint8_t* w13,
                          const uint8_t* w13_sc, const uint8_t* w2, const uint8_t* w2_sc, int I, bool fp4mid, void* y,
                          bool bf16_out, void* ws, hipStream_t stream, const char** variant) {
  float* h = static_cast<float*>(ws);
  uint8_t* q = static_cast<uint8_t*>(ws) + a256((size_t)T * 2 * I * 4);
  uint8_t* q_sc = q + a256((size_t)T * (fp4mid ? I / 2 : I));
  hipError_t e = launch_fp4_gemm(x, x_sc, fp4x, w13, w13_sc, T, 2 * I, H, h, false, stream, variant);
  if (e != hipSuccess) return e;
  e = launch_swiglu_quantize(h, false, 2 * (int64_t)I, T, I, fp4mid, q, q_sc, stream);
  if (e != hipSuccess) return e;
  e = launch_fp4_gemm(q, q_sc, fp4mid, w2, w2_sc, T, H, I, y, bf16_out, stream, variant);
  *variant = "fp4_ffn:product+swiglu_quantize+product";
  return e;
}

}  // namespace mx
