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
// One wavefront per row up to H = 1024, four up to 4096, eight beyond, the row in registers (chunks of 8 elements per
// lane, all of a row's loads in flight at once, one pass over memory); four neighbouring lanes hold a block of 32, so its
// amax is two quad exchanges.  The split depends on H alone, and with it the order of the sum: a row's bits never depend
// on T.  One wavefront / four per row, us, bf16 rows and residual to h and E4M3 codes: 16 x 512 3.3 / 3.3, 8192 x 512 7.8 / 11.5;
// 16 x 1024 4.0 / 3.4, 8192 x 1024 13.4 / 15.6; 16 x 2048 5.4 / 3.3, 8192 x 2048 24.1 / 21.8.
//
// 8192 x 4096 bf16 with residual, to h, n and E4M3 codes: 50 to 53 us (303 MB, 5.7 to 6.0 TB/s, bound by memory), to h and
// codes alone 37 us (236 MB, 6.3 TB/s); 48 x 5120 4.4 us, one row of 4096 4.0 us (a launch, one round to memory, one
// reduction).
#include "mx_cast.hpp"
#include "mx_launch.hpp"

namespace mx {

// 8 elements as they lie in memory: 16 bytes of bf16 or 32 of fp32
struct Raw8 { u32x4 a, b; };
__device__ __forceinline__ Raw8 raw8(const void* p, bool bf16, int64_t i) {
  Raw8 r;
  if (bf16) {
    r.a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
    r.b = u32x4{0, 0, 0, 0};
  } else {
    const u32x4* s = reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + i);
    r.a = s[0];
    r.b = s[1];
  }
  return r;
}
__device__ __forceinline__ void values8(const Raw8& r, bool bf16, float* v) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t h = r.a[j / 2];
    const uint32_t w = bf16 ? ((j & 1) ? h & 0xFFFF0000u : h << 16) : (j < 4 ? r.a[j & 3] : r.b[j & 3]);
    v[j] = __uint_as_float(w);
  }
}

template <int WAVES, int NCH, bool X16, bool R16>
__global__ __launch_bounds__(WAVES > 4 ? 64 * WAVES : 256) void add_rmsnorm_kernel(NormArgs A, int T) {
  __shared__ double part[WAVES];
  constexpr int LANES = 64 * WAVES;                               // of one row
  const int tid = threadIdx.x % LANES, nch = A.H / 8;
  const int64_t t = WAVES == 1 ? (int64_t)blockIdx.x * 4 + threadIdx.x / 64 : blockIdx.x;
  if (WAVES == 1 && t >= T) return;
  const bool has_r = A.residual != nullptr, has_x2 = A.x2 != nullptr;
  Raw8 x[NCH], r[NCH], x2[NCH];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {                                 // lanes past the row read its last chunk again
    const int ch = min(c * LANES + tid, nch - 1);
    x[c] = raw8(A.x, X16, t * A.x_ld + ch * 8);
    if (has_r) r[c] = raw8(A.residual, R16, t * A.r_ld + ch * 8);
    if (has_x2) x2[c] = raw8(A.x2, X16, t * A.x_ld + ch * 8);
  }
  float v[NCH][8];
  double ss[2] = {0.0, 0.0};
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    float a[8];
    values8(x[c], X16, v[c]);
    if (has_r) {
      values8(r[c], R16, a);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = a[j] + v[c][j];
    }
    if (has_x2) {
      values8(x2[c], X16, a);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = v[c][j] + a[j];
    }
    if (R16 && (has_r || A.h)) {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const uint32_t d = bf16_pair(v[c][j], v[c][j + 1]);
        v[c][j] = __uint_as_float(d << 16);
        v[c][j + 1] = __uint_as_float(d & 0xFFFF0000u);
      }
    }
    if (c * LANES + tid < nch) {
#pragma unroll
      for (int j = 0; j < 8; ++j) ss[j & 1] = fma((double)v[c][j], (double)v[c][j], ss[j & 1]);
    }
  }
  double sum = ss[0] + ss[1];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  if (WAVES > 1) {
    if ((tid & 63) == 0) part[tid >> 6] = sum;
    __syncthreads();
    sum = part[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) sum += part[w];
  }
  const double rr = rsqrt(sum * A.inv_h + (double)A.eps);
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int ch = c * LANES + tid;
    if (ch < nch) {                               // whole blocks of 32 (four lanes) are in or out: H % 32 == 0
      if (A.h) store8(A.h, R16, t * A.r_ld + ch * 8, v[c]);
      float w[8];
      if (A.w) load8(A.w, A.w_bf16, ch * 8, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = (float)((double)v[c][j] * rr * (A.w ? (double)w[j] : 1.0));
      if (A.n) store8(A.n, true, t * A.H + ch * 8, v[c]);
      if (A.q) {
        if (A.fp4) store8_codes<true>(v[c], A.q, A.sc, t * nch + ch);
        else store8_codes<false>(v[c], A.q, A.sc, t * nch + ch);
      }
    }
  }
}

template <int WAVES, int NCH>
static void launch_norm(const NormArgs& a, int T, hipStream_t stream) {
  const dim3 grid(WAVES == 1 ? (unsigned)(((int64_t)T + 3) / 4) : (unsigned)T), block(WAVES > 4 ? 64 * WAVES : 256);
  if (a.x_bf16 && a.r_bf16) hipLaunchKernelGGL((add_rmsnorm_kernel<WAVES, NCH, true, true>), grid, block, 0, stream, a, T);
  else if (a.x_bf16) hipLaunchKernelGGL((add_rmsnorm_kernel<WAVES, NCH, true, false>), grid, block, 0, stream, a, T);
  else if (a.r_bf16) hipLaunchKernelGGL((add_rmsnorm_kernel<WAVES, NCH, false, true>), grid, block, 0, stream, a, T);
  else hipLaunchKernelGGL((add_rmsnorm_kernel<WAVES, NCH, false, false>), grid, block, 0, stream, a, T);
}

hipError_t launch_add_rmsnorm(const NormArgs& a, int T, hipStream_t stream) {
  if (a.H <= 512) launch_norm<1, 1>(a, T, stream);
  else if (a.H <= 1024) launch_norm<1, 2>(a, T, stream);
  else if (a.H <= 2048) launch_norm<4, 1>(a, T, stream);
  else if (a.H <= 4096) launch_norm<4, 2>(a, T, stream);
  else if (a.H <= 8192) launch_norm<8, 2>(a, T, stream);
  else launch_norm<8, 4>(a, T, stream);
  return hipGetLastError();
}

}  // namespace mx
