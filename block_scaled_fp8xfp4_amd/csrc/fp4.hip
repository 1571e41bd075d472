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

// Many rows: BM x BN output tiles staged through LDS.  A stage holds K = 128
// of the tile's activation rows, weight rows and scale dwords, brought by LDS
// DMA NST stages ahead of the matrix cores and ordered by vmcnt waits and
// LDS-only barriers, one barrier per stage.  Inside a stage two steps of
// 32x32x64, the shape in which E2M1 x E2M1 runs at its full rate; the next
// step's operands are read from LDS while the current one multiplies, across
// the stage's barrier too.
//
// The weights take the instruction's A side and the activations its B side,
// so a lane holds one row of y and four consecutive columns per register
// quad: lane l has row l % 32 and columns 8 q + 4 (l / 32) + [0, 4), q = 0..3.
//
// LDS rows are 64 bytes (E2M1) or 128 (E4M3) in 16-byte chunks; the chunk
// index is XORed with bits of the row so that 8 (and 16) consecutive rows'
// reads of one chunk fall on different banks.
typedef float v16f __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2_a4 __attribute__((ext_vector_type(2), aligned(4)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ int swz4(int r) { return (((r >> 1) ^ (r >> 3)) & 1) | ((r >> 1) & 2); }
__device__ __forceinline__ int swz8(int r) { return ((r >> 1) & 3) | (((r ^ (r >> 3)) & 1) << 2); }

__device__ __forceinline__ u32x4 lds_read16(uint32_t addr) {
  return *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(addr);
}
__device__ __forceinline__ uint32_t lds_read4(uint32_t addr) {
  return *reinterpret_cast<const __attribute__((address_space(3))) uint32_t*>(addr);
}
__device__ __forceinline__ v8i operand(const u32x4& lo) {
  return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], 0, 0, 0, 0};
}
__device__ __forceinline__ v8i operand(const u32x4& lo, const u32x4& hi) {
  return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

template <int V> struct Int { static constexpr int value = V; };

constexpr int KS = 128;                           // K per stage
constexpr int XCDS = 8;

// WM x WN wavefronts of TM x TN 32 x 32 tiles each.
template <bool FP4A, int WM, int WN, int TM, int TN, int NST>
struct TileShape {
  static constexpr int NW = WM * WN, BM = WM * TM * 32, BN = WN * TN * 32;
  static constexpr int RA = FP4A ? KS / 2 : KS;   // bytes of an activation row per stage
  static constexpr int CA = RA / 16;              // its chunks
  static constexpr uint32_t OFF_W = BM * RA, OFF_XS = OFF_W + BN * (KS / 2), OFF_WS = OFF_XS + BM * 4;
  static constexpr uint32_t STAGE = OFF_WS + BN * 4;
  static constexpr int NX = BM * RA / 1024 / NW, NWT = BN * (KS / 2) / 1024 / NW;   // DMA instructions per wavefront
  static constexpr int NSC = ((BM + BN) / 64 + NW - 1) / NW;
  static constexpr int NV = NX + NWT + NSC;       // vector-memory operations per wavefront and stage
  static_assert(NX * NW * 1024 == BM * RA && NWT * NW * 1024 == BN * (KS / 2), "whole DMA instructions");
  static_assert(STAGE * NST <= 160 * 1024 && NV * (NST - 1) < 63, "LDS and vmcnt");
};

template <int N> __device__ __forceinline__ void wait_vm() { asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory"); }

// at most `left` (0 .. NST - 1) whole stages may still be in flight
template <int NV, int NST> __device__ __forceinline__ void wait_stages(int left) {
  if (NST > 3 && left >= 3) wait_vm<3 * NV>();
  else if (NST > 2 && left >= 2) wait_vm<2 * NV>();
  else if (left >= 1) wait_vm<NV>();
  else wait_vm<0>();
}

template <bool FP4A, int WM, int WN, int TM, int TN, int NST, bool TAIL>
__global__ __launch_bounds__(64 * WM * WN, 2) void fp4_tile_kernel(const uint8_t* __restrict__ a, const uint8_t* __restrict__ a_sc,
                                                                   const uint8_t* __restrict__ w, const uint8_t* __restrict__ w_sc,
                                                                   int M, int N, int K, void* __restrict__ y, bool bf16_out) {
  using S = TileShape<FP4A, WM, WN, TM, TN, NST>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::STAGE * NST];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 31, g = lane >> 5;
  const int wm = wave / WN, wn = wave % WN;
  const int nblk = K / 32, ns = (K + KS - 1) / KS;
  const int rowa = FP4A ? K / 2 : K, roww = K / 2;

  // XCD-aware order: each XCD takes a run of consecutive tiles, which go down 8 row tiles before the next column tile
  const int nrt = (M + S::BM - 1) / S::BM, nct = (N + S::BN - 1) / S::BN;
  const int64_t tiles = (int64_t)nrt * nct, per = (tiles + XCDS - 1) / XCDS;
  const int64_t t = (int64_t)(blockIdx.x % XCDS) * per + blockIdx.x / XCDS;
  if (t >= tiles) return;
  const int grp = (int)(t / (8 * (int64_t)nct)), in = (int)(t - grp * 8 * (int64_t)nct);
  const int rows_in = min(8, nrt - grp * 8);
  const int rt = grp * 8 + in % rows_in, ct = in / rows_in;
  const int64_t m0 = (int64_t)rt * S::BM, n0 = (int64_t)ct * S::BN;
  const int mlast = (int)(M - 1 - m0), nlast = (int)(N - 1 - n0);   // rows past the end repeat the last one

  // this lane's DMA sources: byte offsets from the tile's first row
  uint32_t xoff[S::NX], woff[S::NWT], xc[S::NX], wc[S::NWT], soff[S::NSC];
#pragma unroll
  for (int i = 0; i < S::NX; ++i) {
    const int p = (i * S::NW + wave) * 64 + lane, r = p / S::CA;
    const int c = (p % S::CA) ^ (FP4A ? swz4(r) : swz8(r));
    xc[i] = c * (FP4A ? 32 : 16);
    xoff[i] = (uint32_t)min(r, mlast) * (uint32_t)rowa + c * 16;
  }
#pragma unroll
  for (int i = 0; i < S::NWT; ++i) {
    const int p = (i * S::NW + wave) * 64 + lane, r = p / 4, c = (p % 4) ^ swz4(r);
    wc[i] = c * 32;
    woff[i] = (uint32_t)min(r, nlast) * (uint32_t)roww + c * 16;
  }
  int sslot[S::NSC];
#pragma unroll
  for (int i = 0; i < S::NSC; ++i) {
    sslot[i] = min(i * S::NW + wave, (S::BM + S::BN) / 64 - 1);      // surplus wavefronts repeat the last slot
    const int r = sslot[i] * 64 + lane;
    soff[i] = (uint32_t)(sslot[i] < S::BM / 64 ? min(r, mlast) : min(r - S::BM, nlast)) * (uint32_t)nblk;
  }
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(lds));
  const uint8_t* at = a + m0 * rowa;
  const uint8_t* wt = w + n0 * roww;
  const uint8_t* ast = a_sc + m0 * nblk;
  const uint8_t* wst = w_sc + n0 * nblk;
  auto issue = [&](int s, uint32_t base) {
    const bool cut = TAIL && s == ns - 1;                             // chunks past K read the stage's first chunk
#pragma unroll
    for (int i = 0; i < S::NX; ++i) {
      const uint32_t off = cut && s * KS + (int)xc[i] >= K ? xoff[i] - xc[i] / (FP4A ? 2 : 1) : xoff[i];
      dma16_to_lds(at + (int64_t)s * S::RA, off, base + (i * S::NW + wave) * 1024);
    }
#pragma unroll
    for (int i = 0; i < S::NWT; ++i) {
      const uint32_t off = cut && s * KS + (int)wc[i] >= K ? woff[i] - wc[i] / 2 : woff[i];
      dma16_to_lds(wt + (int64_t)s * (KS / 2), off, base + S::OFF_W + (i * S::NW + wave) * 1024);
    }
    if (!TAIL) {
#pragma unroll
      for (int i = 0; i < S::NSC; ++i)
        dma4_to_lds((sslot[i] < S::BM / 64 ? ast : wst) + s * 4, soff[i], base + S::OFF_XS + sslot[i] * 256);
    }
  };

  // Operands of one step, and the scale dwords of a stage shifted so that bytes 0 and 2 are the blocks of this lane's
  // half in steps 0 and 1.
  struct Regs { u32x4 xlo[TM], xhi[FP4A ? 1 : TM], w[TN]; };
  struct Scales { uint32_t x[TM], w[TN]; };
  const uint32_t xrow = (uint32_t)(wm * TM * 32 + lr), wrow = (uint32_t)(wn * TN * 32 + lr);
  const int fx = FP4A ? swz4(lr) : swz8(lr), fw = swz4(lr);
  constexpr int NLD = TN + TM * (FP4A ? 1 : 2), NMM = TM * TN;       // LDS reads and matrix operations of a step
  // the it-th LDS read of step ks (weights first: every matrix operation row needs them)
  auto load1 = [&](Regs& R, uint32_t base, int ks, int it) {
    if (it < TN) R.w[it] = lds_read16(base + S::OFF_W + wrow * 64 + ((2 * ks + g) ^ fw) * 16 + it * 2048);
    else if (FP4A) R.xlo[it - TN] = lds_read16(base + xrow * S::RA + ((2 * ks + g) ^ fx) * 16 + (it - TN) * 32 * S::RA);
    else {
      const int i = (it - TN) / 2;
      if ((it - TN) % 2 == 0) R.xlo[i] = lds_read16(base + xrow * S::RA + ((4 * ks + g) ^ fx) * 16 + i * 32 * S::RA);
      else R.xhi[i] = lds_read16(base + xrow * S::RA + ((4 * ks + 2 + g) ^ fx) * 16 + i * 32 * S::RA);
    }
  };
  auto load_scales = [&](Scales& C, uint32_t base) {
#pragma unroll
    for (int i = 0; i < TM; ++i) C.x[i] = lds_read4(base + S::OFF_XS + (xrow + i * 32) * 4);
#pragma unroll
    for (int i = 0; i < TN; ++i) C.w[i] = lds_read4(base + S::OFF_WS + (wrow + i * 32) * 4);
  };
  auto shift_scales = [&](Scales& C) {
#pragma unroll
    for (int i = 0; i < TM; ++i) C.x[i] >>= 8 * g;
#pragma unroll
    for (int i = 0; i < TN; ++i) C.w[i] >>= 8 * g;
  };
  v16f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  auto cut_step = [&](Regs& R, int s, int ks) {                       // zero elements past K (activations; E2M1 weights are finite)
    const int b = s * 4 + 2 * ks;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      if (b + (FP4A ? g : 0) >= nblk) R.xlo[i] = u32x4{0, 0, 0, 0};
      if (!FP4A && b + 1 >= nblk) R.xhi[FP4A ? 0 : i] = u32x4{0, 0, 0, 0};
    }
  };
  auto mma = [&](const Regs& R, const Scales& C, auto step, int q) {   // the q-th matrix operation of step `step`
    constexpr int B = 2 * decltype(step)::value;
    const int i = q / TN, j = q % TN;
    const v8i xv = FP4A ? operand(R.xlo[i]) : operand(R.xlo[i], R.xhi[FP4A ? 0 : i]);
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(R.w[j]), xv, acc[i][j], 4, FP4A ? 4 : 0, B,
                                                                (int)C.w[j], B, (int)C.x[i]);
  };
  // One step's matrix operations with the next step's LDS reads between them (the order is held by scheduling barriers).
  auto step_with_loads = [&](const Regs& R, const Scales& C, auto step, Regs& Rn, uint32_t base, int ks) {
#pragma unroll
    for (int q = 0; q < NMM; ++q) {
#pragma unroll
      for (int it = q * NLD / NMM; it < (q + 1) * NLD / NMM; ++it) load1(Rn, base, ks, it);
      mma(R, C, step, q);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  const Int<0> Step0;
  const Int<1> Step1;

  // K % 128 != 0: scale rows are not dword-aligned; each lane keeps its slots' next dword in registers and writes it
  // to the stage's LDS before the barrier that publishes the stage (bytes past K: 127)
  uint32_t sreg[S::NSC];
  auto fetch_scales = [&](int s) {
#pragma unroll
    for (int i = 0; i < S::NSC; ++i) {
      const uint8_t* p = (sslot[i] < S::BM / 64 ? ast : wst) + soff[i] + s * 4;
      uint32_t v = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) v |= (uint32_t)(s * 4 + b < nblk ? p[b] : 127) << (8 * b);
      sreg[i] = v;
    }
  };
  auto put_scales = [&](uint32_t base) {
#pragma unroll
    for (int i = 0; i < S::NSC; ++i)
      *reinterpret_cast<__attribute__((address_space(3))) uint32_t*>(base + S::OFF_XS + sslot[i] * 256 + lane * 4) = sreg[i];
  };

#pragma unroll
  for (int s = 0; s < NST; ++s)
    if (s < ns) issue(s, lds0 + s * S::STAGE);
  if (TAIL) {
    fetch_scales(0);
    put_scales(lds0);
    if (ns > 1) fetch_scales(1);
  }
  if (TAIL) wait_vm<0>();
  else wait_stages<S::NV, NST>(min(ns - 1, NST - 1));
  lds_barrier();
  Regs R0, R1;
  Scales C, Cn;
#pragma unroll
  for (int it = 0; it < NLD; ++it) load1(R0, lds0, 0, it);
  load_scales(C, lds0);
  shift_scales(C);
  if (TAIL && ns == 1) cut_step(R0, 0, 0);
  uint32_t b0 = lds0;
  // Stage s: step 0 while step 1's operands are read; then the next stage's data is waited for and published, this
  // stage's buffer (read out by every wavefront) refilled, and step 1 multiplies while the next stage's are read.
  auto stage = [&](int s, auto refill) {
    const uint32_t b1 = b0 + S::STAGE == lds0 + NST * S::STAGE ? lds0 : b0 + S::STAGE;
    step_with_loads(R0, C, Step0, R1, b0, 1);
    if (TAIL) {
      put_scales(b1);
      wait_vm<0>();
    } else if (decltype(refill)::value) {
      wait_vm<S::NV * (NST - 2)>();
    } else {
      wait_stages<S::NV, NST>(min(ns - 2 - s, NST - 2));
    }
    lds_barrier();
    if (decltype(refill)::value) issue(s + NST, b0);
    if (TAIL && s + 2 < ns) fetch_scales(s + 2);
    load_scales(Cn, b1);
    __builtin_amdgcn_sched_barrier(0);
    step_with_loads(R1, C, Step1, R0, b1, 0);
    if (TAIL && s + 1 == ns - 1) cut_step(R0, s + 1, 0);
    shift_scales(Cn);
    C = Cn;
    b0 = b1;
  };
  int s = 0;
  for (; s + NST < ns; ++s) stage(s, Step1);
  for (; s + 1 < ns; ++s) stage(s, Step0);
#pragma unroll
  for (int it = 0; it < NLD; ++it) load1(R1, b0, 1, it);
  if (TAIL) cut_step(R1, s, 1);
#pragma unroll
  for (int q = 0; q < NMM; ++q) mma(R0, C, Step0, q);
#pragma unroll
  for (int q = 0; q < NMM; ++q) mma(R1, C, Step1, q);

  const bool quads = (N & 3) == 0;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t m = m0 + wm * TM * 32 + i * 32 + lr;
    if (m >= M) continue;
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t n = n0 + wn * TN * 32 + j * 32 + 8 * q + 4 * g;
        const float v0 = acc[i][j][4 * q], v1 = acc[i][j][4 * q + 1], v2 = acc[i][j][4 * q + 2], v3 = acc[i][j][4 * q + 3];
        if (quads) {
          if (n >= N) continue;
          if (bf16_out) {
            const u32x2_a4 d = {(uint32_t)f32_to_bf16_rne(v0) | ((uint32_t)f32_to_bf16_rne(v1) << 16),
                                (uint32_t)f32_to_bf16_rne(v2) | ((uint32_t)f32_to_bf16_rne(v3) << 16)};
            *reinterpret_cast<u32x2_a4*>(static_cast<uint16_t*>(y) + m * N + n) = d;
          } else {
            *reinterpret_cast<f32x4_a4*>(static_cast<float*>(y) + m * N + n) = f32x4_a4{v0, v1, v2, v3};
          }
        } else {
          const float v[4] = {v0, v1, v2, v3};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < N) {
              if (bf16_out) static_cast<uint16_t*>(y)[m * N + n + e] = f32_to_bf16_rne(v[e]);
              else static_cast<float*>(y)[m * N + n + e] = v[e];
            }
        }
      }
  }
}

constexpr int FP4_TILE_MIN_M = 64;

template <bool FP4A, int WM, int WN, int TM, int TN, int NST>
static void launch_tile(const uint8_t* a, const uint8_t* a_sc, const uint8_t* w, const uint8_t* w_sc, int M, int N, int K,
                        void* y, bool bf16_out, hipStream_t stream) {
  using S = TileShape<FP4A, WM, WN, TM, TN, NST>;
  const int64_t tiles = (int64_t)((M + S::BM - 1) / S::BM) * ((N + S::BN - 1) / S::BN);
  const dim3 grid((unsigned)((tiles + XCDS - 1) / XCDS * XCDS)), block(64 * S::NW);
  if (K % KS) hipLaunchKernelGGL((fp4_tile_kernel<FP4A, WM, WN, TM, TN, NST, true>), grid, block, 0, stream, a, a_sc, w, w_sc, M, N, K, y, bf16_out);
  else hipLaunchKernelGGL((fp4_tile_kernel<FP4A, WM, WN, TM, TN, NST, false>), grid, block, 0, stream, a, a_sc, w, w_sc, M, N, K, y, bf16_out);
}

hipError_t launch_fp4_gemm(const uint8_t* a, const uint8_t* a_sc, bool fp4a, const uint8_t* w, const uint8_t* w_sc,
                           int M, int N, int K, void* y, bool bf16_out, hipStream_t stream, const char** variant) {
  if (M >= FP4_TILE_MIN_M) {
    const int64_t big = (int64_t)((M + 255) / 256) * ((N + 255) / 256);
    if (big >= 192) {
      if (fp4a) launch_tile<true, 2, 4, 4, 2, 4>(a, a_sc, w, w_sc, M, N, K, y, bf16_out, stream);
      else launch_tile<false, 4, 2, 2, 4, 3>(a, a_sc, w, w_sc, M, N, K, y, bf16_out, stream);
      *variant = fp4a ? "fp4:tile256x256_a4" : "fp4:tile256x256_a8";
    } else {
      if (fp4a) launch_tile<true, 2, 2, 2, 2, 4>(a, a_sc, w, w_sc, M, N, K, y, bf16_out, stream);
      else launch_tile<false, 2, 2, 2, 2, 3>(a, a_sc, w, w_sc, M, N, K, y, bf16_out, stream);
      *variant = fp4a ? "fp4:tile128x128_a4" : "fp4:tile128x128_a8";
    }
    return hipGetLastError();
  }
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
