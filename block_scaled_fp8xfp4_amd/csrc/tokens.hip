// Tokens to the order of their experts and back (the buckets of moe_route):
//   permute:        out[slot_pos[t][j]] = x[t]
//   unpermute:      y[t] = sum_j w[t][j] * o[slot_pos[t][j]], fp32, in slot order
//   unpermute_grad: d_o[slot_pos[t][j]] = w[t][j] * dy[t],  dw[t][j] = <dy[t], o[slot_pos[t][j]]>
// A slot that is nowhere (slot_pos < 0 or past the rows there are) takes no
// part.  All of it is memory traffic; every result has one writer and a fixed
// order of addition, so nothing depends on timing.
#include "any_device.hpp"
#include "b128_launch.hpp"

namespace mx {

// More than 64 MB go past the caches, where the step that reads them would not find them all, and the experts' rows are
// loaded so that the caches do not keep them: 8192 x 8 rows of 8 KB are sorted in 103 us from 119, brought back in 104 from
// 123, and their gradient made in 227 from 240.
static bool far_bytes(int64_t n) { return n > int64_t(64) << 20; }

// ---------------------------------------------------------------------------
// Rows of bytes: a thread holds 16 bytes of a token's row (or of its scales)
// and writes them to the token's k places, so that each row is read once.  A
// row's last piece reaches back to be whole (two threads then write the same
// bytes); rows of less than 16 bytes go by bytes.
int64_t permute_chunks(int64_t row, int64_t sc) { return (row + 15) / 16 + (sc + 15) / 16; }

template <bool FAR>
__global__ __launch_bounds__(256) void permute_kernel(PermuteArgs A, uint32_t chunks, uint32_t row_chunks, uint32_t n) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= n) return;
  const uint32_t t = i / chunks, c = i - t * chunks;
  const bool scales = c >= row_chunks;
  const uint8_t* src = scales ? A.x_sc + (int64_t)t * A.sc : A.x + (int64_t)t * A.x_ld;
  uint8_t* const dst = scales ? A.out_sc : A.out;
  const int64_t len = scales ? A.sc : A.row;
  const int64_t at = (int64_t)(scales ? c - row_chunks : c) * 16;
  const int32_t* pos = A.slot_pos + (int64_t)t * A.k;
  if (len >= 16) {
    const int64_t b = min(at, len - 16);
    const u32x4 v = *reinterpret_cast<const u32x4_a1*>(src + b);
    for (int j = 0; j < A.k; ++j) {
      const int p = pos[j];
      if (p < 0 || p >= A.out_rows) continue;
      u32x4_a1* const to = reinterpret_cast<u32x4_a1*>(dst + (int64_t)p * len + b);
      if constexpr (FAR) __builtin_nontemporal_store(v, to);
      else *to = v;
    }
    return;
  }
  for (int j = 0; j < A.k; ++j) {
    const int p = pos[j];
    if (p < 0 || p >= A.out_rows) continue;
    for (int64_t b = 0; b < len; ++b) dst[(int64_t)p * len + b] = src[b];
  }
}

hipError_t launch_permute(const PermuteArgs& a, hipStream_t stream) {
  const int64_t chunks = permute_chunks(a.row, a.sc), n = a.T * chunks;
  if (n == 0 || a.k == 0) return hipSuccess;
  const dim3 grid((unsigned)((n + 255) / 256));
  const uint32_t row_chunks = (uint32_t)((a.row + 15) / 16);
  if (far_bytes((int64_t)a.T * a.k * (a.row + a.sc))) hipLaunchKernelGGL(permute_kernel<true>, grid, dim3(256), 0, stream, a, (uint32_t)chunks, row_chunks, (uint32_t)n);
  else hipLaunchKernelGGL(permute_kernel<false>, grid, dim3(256), 0, stream, a, (uint32_t)chunks, row_chunks, (uint32_t)n);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// A thread per N columns of a token; a row's last piece reaches back to be whole (N = 1 for rows of less than 8).
template <int N, bool OB, bool YB, bool FAR>
__global__ __launch_bounds__(256) void unpermute_kernel(UnpermuteArgs A, uint32_t chunks, uint32_t n) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= n) return;
  const uint32_t t = i / chunks;
  const int c = min((int)(i - t * chunks) * N, A.H - N);
  const int32_t* pos = A.slot_pos + (int64_t)t * A.k;
  const float* w = A.w + (int64_t)t * A.k;
  float acc[N];
#pragma unroll
  for (int e = 0; e < N; ++e) acc[e] = 0.0f;
  constexpr int AT = 4;                                      // slots whose rows are on their way at a time
  for (int j0 = 0; j0 < A.k; j0 += AT) {
    int p[AT];
    float f[AT], v[AT][N];
#pragma unroll
    for (int j = 0; j < AT; ++j) {
      p[j] = j0 + j < A.k ? pos[j0 + j] : -1;
      f[j] = A.w && j0 + j < A.k ? w[j0 + j] : 1.0f;
    }
#pragma unroll
    for (int j = 0; j < AT; ++j)
      if (p[j] >= 0 && p[j] < A.o_rows) load_any<N, true>(A.o, OB, (int64_t)p[j] * A.H + c, v[j]);
#pragma unroll
    for (int j = 0; j < AT; ++j) {
      if (p[j] < 0 || p[j] >= A.o_rows) continue;
#pragma unroll
      for (int e = 0; e < N; ++e) acc[e] = __builtin_fmaf(f[j], v[j][e], acc[e]);
    }
  }
  store_any<N, FAR>(A.y, YB, (int64_t)t * A.H + c, acc);
}

template <int N, bool OB, bool FAR> static void launch_unpermute_of(const UnpermuteArgs& a, hipStream_t stream) {
  const int64_t chunks = (a.H + N - 1) / N, n = a.T * chunks;
  const dim3 grid((unsigned)((n + 255) / 256));
  if (a.y_bf16) hipLaunchKernelGGL((unpermute_kernel<N, OB, true, FAR>), grid, dim3(256), 0, stream, a, (uint32_t)chunks, (uint32_t)n);
  else hipLaunchKernelGGL((unpermute_kernel<N, OB, false, FAR>), grid, dim3(256), 0, stream, a, (uint32_t)chunks, (uint32_t)n);
}
hipError_t launch_unpermute(const UnpermuteArgs& a, hipStream_t stream) {
  if (a.H < 8) {
    if (a.o_bf16) launch_unpermute_of<1, true, false>(a, stream);
    else launch_unpermute_of<1, false, false>(a, stream);
  } else if (far_bytes((int64_t)a.T * a.k * a.H * (a.o_bf16 ? 2 : 4))) {
    if (a.o_bf16) launch_unpermute_of<8, true, true>(a, stream);
    else launch_unpermute_of<8, false, true>(a, stream);
  } else {
    if (a.o_bf16) launch_unpermute_of<8, true, false>(a, stream);
    else launch_unpermute_of<8, false, false>(a, stream);
  }
  return hipGetLastError();
}

// A wavefront per (token, slot): it scales the token's dy into the slot's row of d_o and sums dy * o on the way, eight
// columns a lane.  d_o may be o itself: a lane has read a piece before it writes it.
template <bool DYB, bool OB, bool FAR>
__global__ __launch_bounds__(256) void unpermute_grad_kernel(UnpermuteArgs A) {
  const int lane = threadIdx.x & 63;
  const int64_t pair = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (pair >= (int64_t)A.T * A.k) return;
  const int64_t t = pair / A.k;
  const int p = A.slot_pos[pair];
  if (p < 0 || p >= A.o_rows) {
    if (A.dw && lane == 0) A.dw[pair] = 0.0f;
    return;
  }
  const float f = A.w ? A.w[pair] : 1.0f;
  const int64_t dy0 = t * A.H, o0 = (int64_t)p * A.H;
  float sum = 0.0f;
  // B pieces of N columns, `apart` columns apart, those before the row's end, all on their way at a time
  auto pieces = [&](auto size, auto batch, int c, int apart, int end) {
    constexpr int N = decltype(size)::value, B = decltype(batch)::value;
    float d[B][N], v[B][N];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      if (c + b * apart >= end) continue;
      load_any<N>(A.y, DYB, dy0 + c + b * apart, d[b]);
      if (A.dw) load_any<N, true>(A.o, OB, o0 + c + b * apart, v[b]);
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      if (c + b * apart >= end) continue;
      if (A.dw) {
#pragma unroll
        for (int e = 0; e < N; ++e) sum = __builtin_fmaf(d[b][e], v[b][e], sum);
      }
      if (!A.d_o) continue;
#pragma unroll
      for (int e = 0; e < N; ++e) d[b][e] *= f;
      store_any<N, FAR>(A.d_o, OB, o0 + c + b * apart, d[b]);
    }
  };
  const int whole = A.H & ~7;
  for (int c = lane * 8; c < whole; c += 1024) pieces(Int<8>{}, Int<2>{}, c, 512, whole);
  pieces(Int<1>{}, Int<1>{}, whole + lane, 1, A.H);
  if (!A.dw) return;
#pragma unroll
  for (int d = 32; d >= 1; d /= 2) sum += __shfl_xor(sum, d);
  if (lane == 0) A.dw[pair] = sum;
}

template <bool DYB, bool OB> static void launch_unpermute_grad_of(const UnpermuteArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)(((int64_t)a.T * a.k + 3) / 4)), block(256);
  if (far_bytes((int64_t)a.T * a.k * a.H * (OB ? 2 : 4))) hipLaunchKernelGGL((unpermute_grad_kernel<DYB, OB, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((unpermute_grad_kernel<DYB, OB, false>), grid, block, 0, stream, a);
}
hipError_t launch_unpermute_grad(const UnpermuteArgs& a, hipStream_t stream) {
  if (a.y_bf16) {
    if (a.o_bf16) launch_unpermute_grad_of<true, true>(a, stream);
    else launch_unpermute_grad_of<true, false>(a, stream);
  } else {
    if (a.o_bf16) launch_unpermute_grad_of<false, true>(a, stream);
    else launch_unpermute_grad_of<false, false>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace mx
