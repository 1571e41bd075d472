// Residual addition + root-mean-square norm + block-32 codes, the kernel between two layers: it makes the rows that the
// library's layers read (the router's bf16 hidden rows, the E4M3 / E2M1 codes and scales of the experts and of the dense
// products) from what they wrote (fp32 or bf16) and the residual stream ("New Deepseek 4.1 flash recipe" thread, post #6,
// "Kernel by kernel against B12X": the step's quantization + norms group).
//
//   v = (residual + x) + x2 in fp32;  h = v rounded to the residual's type (stored)
//   r = 1 / sqrt(sum h^2 / H + eps);  n = fp32((h * r) * w);  outputs: h, bf16(n), codes(n)
//
// The sum, r and the products run in double, rounded once to fp32: a code then depends on h and w alone, not on the order
// of a 32-bit sum (with an error of 1e-7 in r, a few codes per million land on the other side of a rounding border).  At 8
// double operations per element that is far under the memory time.  The norm reads h as stored, so the fused call equals
// the addition, then the norm of what it wrote.
//
// One workgroup of 256 threads per row, the row in registers (chunks of 8 elements per thread, one pass over memory); four
// neighbouring lanes hold a block of 32, so its amax is two quad exchanges.  The split depends on H alone, and with it the
// order of the sum: a row's bits never depend on T.
#include "mx_device.hpp"
#include "mx_launch.hpp"

namespace mx {

template <int NCH>
__global__ __launch_bounds__(256) void add_rmsnorm_kernel(NormArgs A) {
  __shared__ double part[4];
  const int tid = threadIdx.x, nch = A.H / 8;
  const int64_t t = blockIdx.x;
  float v[NCH][8];
  double ss = 0.0;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int ch = c * 256 + tid;
    if (ch < nch) {
      float a[8];
      load8(A.x, A.x_bf16, t * A.x_ld + ch * 8, v[c]);
      if (A.residual) {
        load8(A.residual, A.r_bf16, t * A.r_ld + ch * 8, a);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] = a[j] + v[c][j];
      }
      if (A.x2) {
        load8(A.x2, A.x_bf16, t * A.x_ld + ch * 8, a);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] = v[c][j] + a[j];
      }
      if ((A.residual || A.h) && A.r_bf16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] = __uint_as_float((uint32_t)f32_to_bf16_rne(v[c][j]) << 16);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fma((double)v[c][j], (double)v[c][j], ss);
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) ss += __shfl_xor(ss, o);
  if ((tid & 63) == 0) part[tid >> 6] = ss;
  __syncthreads();
  const double r = 1.0 / sqrt(((part[0] + part[1]) + (part[2] + part[3])) / (double)A.H + (double)A.eps);
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int ch = c * 256 + tid;
    if (ch < nch) {                               // whole blocks of 32 (four lanes) are in or out: H % 32 == 0
      if (A.h) store8(A.h, A.r_bf16, t * A.r_ld + ch * 8, v[c]);
      float w[8];
      if (A.w) load8(A.w, A.w_bf16, ch * 8, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = (float)((double)v[c][j] * r * (A.w ? (double)w[j] : 1.0));
      if (A.n) store8(A.n, true, t * A.H + ch * 8, v[c]);
      if (A.q) {
        if (A.fp4) store8_codes<true>(v[c], A.q, A.sc, t * nch + ch);
        else store8_codes<false>(v[c], A.q, A.sc, t * nch + ch);
      }
    }
  }
}

hipError_t launch_add_rmsnorm(const NormArgs& a, int T, hipStream_t stream) {
  const dim3 grid((unsigned)T), block(256);
  if (a.H <= 2048) hipLaunchKernelGGL(add_rmsnorm_kernel<1>, grid, block, 0, stream, a);
  else if (a.H <= 4096) hipLaunchKernelGGL(add_rmsnorm_kernel<2>, grid, block, 0, stream, a);
  else if (a.H <= 8192) hipLaunchKernelGGL(add_rmsnorm_kernel<4>, grid, block, 0, stream, a);
  else hipLaunchKernelGGL(add_rmsnorm_kernel<8>, grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace mx
