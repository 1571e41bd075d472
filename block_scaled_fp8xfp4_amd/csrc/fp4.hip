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
//
// What the matrix cores keep of a sum (measured): E4M3 x E2M1 products are
// first added in eights of consecutive K, each product cut toward zero at
// 2^-13 of 2^E, E the largest sum of two operands' exponents among those that
// are not zero; the eights and the accumulator are then joined with 24 bits
// and one more, and rounded to nearest even once per 64 of K.  E2M1 x E2M1
// products fit those bits.  The cut is the instruction's; the routed experts'
// products have it too.
#include "mx_cast.hpp"
#include "mx_launch.hpp"

namespace mx {

// E2M1 (A) x E2M1 (B) step, K = 128.
__device__ __forceinline__ v4f mfma_fp4_fp4(const v8i& a, const v8i& b, v4f c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));
typedef uint32_t u32x4_a1 __attribute__((ext_vector_type(4), aligned(1)));

template <typename V> __device__ __forceinline__ V lds_read(uint32_t addr) {
  return *reinterpret_cast<const __attribute__((address_space(3))) V*>(addr);
}
template <typename V> __device__ __forceinline__ void lds_write(uint32_t addr, const V& v) {
  *reinterpret_cast<__attribute__((address_space(3))) V*>(addr) = v;
}

struct TileArgs {
  const uint8_t* x; const uint8_t* x_sc;          // activations [M][K]
  const uint8_t* w; const uint8_t* w_sc;          // weights [N][K]; SwiGLU: [2N][K], gate rows then up rows
  int M, N, K;
  void* y; bool bf16_out;                         // [M][N]
  uint8_t* q; uint8_t* q_sc; bool fp4mid;         // SwiGLU: codes [M][N] instead
};

constexpr int RPK = 512;                          // K per piece of few rows: four 16x16x128 steps

// This lane's column n of rows r0 .. r0 + 3.
__device__ __forceinline__ void store_rows(const TileArgs& A, const v4f& acc, int64_t r0, int64_t n) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (r0 + i >= A.M) continue;
    if (A.bf16_out) static_cast<uint16_t*>(A.y)[(r0 + i) * A.N + n] = f32_to_bf16_rne(acc[i]);
    else static_cast<float*>(A.y)[(r0 + i) * A.N + n] = acc[i];
  }
}

// Up to 16 rows, 16 columns: one wavefront that reads both operands straight
// to registers.  Lane l serves row / column l % 16; lanes past M or N repeat
// the last row / column, their results are not stored.  K past the last whole
// piece is read with clamped addresses and zeroed, its scales are 127.
template <bool FP4A> struct LonePiece { u32x4 w[4], alo[4], ahi[FP4A ? 1 : 4], ws, as; };

template <bool FP4A>
__device__ __forceinline__ void lone_load(LonePiece<FP4A>& P, const uint8_t* wp, const uint8_t* wsp, const uint8_t* ap,
                                          const uint8_t* asp, int c, int g) {
  P.as = *reinterpret_cast<const u32x4_a1*>(asp + c * 16);
  P.ws = *reinterpret_cast<const u32x4_a1*>(wsp + c * 16);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if (FP4A) P.alo[s] = ldg16(ap + c * 256 + s * 64 + g * 16);
    else {
      P.alo[s] = ldg16(ap + c * 512 + s * 128 + g * 16);
      P.ahi[FP4A ? 0 : s] = ldg16(ap + c * 512 + s * 128 + 64 + g * 16);
    }
    P.w[s] = ldg16(wp + c * 256 + s * 64 + g * 16);
  }
}

// The piece that K ends in: blocks past K are read from the last block and replaced.
template <bool FP4A>
__device__ __forceinline__ void lone_load_tail(LonePiece<FP4A>& P, const uint8_t* wp, const uint8_t* wsp,
                                               const uint8_t* ap, const uint8_t* asp, int c, int g, int nblk) {
  const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int b = c * 16 + s * 4 + g, bc = min(b, nblk - 1);
    const u32x4 w = ldg16(wp + bc * 16);
    P.w[s] = b < nblk ? w : zero;
    P.ws[s] = (b < nblk ? (uint32_t)wsp[bc] : 127u) << (8 * g);
    P.as[s] = (b < nblk ? (uint32_t)asp[bc] : 127u) << (8 * g);
    if (FP4A) {
      const u32x4 a = ldg16(ap + bc * 16);
      P.alo[s] = b < nblk ? a : zero;
    } else {                                                          // halves of 16: K = k0 + 16 g and k0 + 64 + 16 g
      const int k = (c * 4 + s) * KSTEP + 16 * g, K = nblk * 32;
      const u32x4 lo = ldg16(ap + min(k, K - 16)), hi = ldg16(ap + min(k + 64, K - 16));
      P.alo[s] = k < K ? lo : zero;
      P.ahi[FP4A ? 0 : s] = k + 64 < K ? hi : zero;
    }
  }
}

template <bool FP4A>
__device__ __forceinline__ v4f lone_multiply(const LonePiece<FP4A>& P, v4f acc, int g) {
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const v8i w = {(int)P.w[s][0], (int)P.w[s][1], (int)P.w[s][2], (int)P.w[s][3], 0, 0, 0, 0};
    const u32x4 lo = P.alo[s], hi = FP4A ? u32x4{0, 0, 0, 0} : P.ahi[FP4A ? 0 : s];
    const v8i a = {(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
    const uint32_t sa = P.as[s] >> (8 * g), sb = P.ws[s] >> (8 * g);
    acc = FP4A ? mfma_fp4_fp4(a, w, acc, sa, sb) : mfma_fp8_fp4(a, w, acc, sa, sb);
  }
  return acc;
}

// The 16 x 16 tile of rows ap (this lane's row) and columns wp (its column) over all of K.
template <bool FP4A>
__device__ __forceinline__ v4f lone_tile(const uint8_t* ap, const uint8_t* asp, const uint8_t* wp, const uint8_t* wsp,
                                         int K, int g) {
  constexpr int RING = FP4A ? 4 : 3;              // 40 and 56 registers each, and one more of them
  const int nblk = K / 32, whole = K / RPK;
  LonePiece<FP4A> P[RING], T;
  v4f acc = {0.f, 0.f, 0.f, 0.f};
  int c = 0;
  if (whole >= RING) {
#pragma unroll
    for (int r = 0; r < RING; ++r) lone_load(P[r], wp, wsp, ap, asp, r, g);
    for (; c + 2 * RING <= whole; c += RING)
#pragma unroll
      for (int r = 0; r < RING; ++r) {
        acc = lone_multiply(P[r], acc, g);
        lone_load(P[r], wp, wsp, ap, asp, c + RING + r, g);
      }
#pragma unroll
    for (int r = 0; r < RING; ++r) {                                  // the last whole pieces but fewer than RING
      acc = lone_multiply(P[r], acc, g);
      if (c + RING + r < whole) lone_load(P[r], wp, wsp, ap, asp, c + RING + r, g);
    }
    c += RING;
  } else {
#pragma unroll
    for (int r = 0; r + 1 < RING; ++r)
      if (r < whole) lone_load(P[r], wp, wsp, ap, asp, r, g);
  }
  if (K % RPK) lone_load_tail(T, wp, wsp, ap, asp, whole, g, nblk);
#pragma unroll
  for (int r = 0; r + 1 < RING; ++r)
    if (c + r < whole) acc = lone_multiply(P[r], acc, g);
  if (K % RPK) acc = lone_multiply(T, acc, g);
  return acc;
}
// WAVES such wavefronts to a workgroup, each 16 rows further down: one for up to 16 rows, four for more of K < 128, where a
// tile is one piece and has nothing to share.
template <bool FP4A, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void fp4_lone_kernel(TileArgs A) {
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int M = A.M, N = A.N, K = A.K, nblk = K / 32;
  const uint32_t nct = (N + 15) / 16;
  const int64_t n0 = (int64_t)(WAVES == 1 ? blockIdx.x : blockIdx.x % nct) * 16;
  const int64_t m0 = WAVES == 1 ? 0 : ((int64_t)(blockIdx.x / nct) * WAVES + (threadIdx.x >> 6)) * 16;
  if (m0 >= M) return;
  const int64_t n = min(n0 + col, (int64_t)N - 1), m = min(m0 + col, (int64_t)M - 1);
  const v4f acc = lone_tile<FP4A>(A.x + m * (FP4A ? K / 2 : K), A.x_sc + m * nblk, A.w + n * (K / 2), A.w_sc + n * nblk, K, g);
  if (n0 + col < N) store_rows(A, acc, m0 + 4 * g, n);
}

// The same for long rows or many columns: workgroups of four wavefronts, all
// of which bring up to 16 rows and their scales to LDS by DMA; CW of them then
// take 16 columns each, whose weights go straight to registers, eight pieces
// of K = 512 in flight.  The weights are asked for behind the rows and before
// the wait for them.  Read by every wavefront, the rows were two thirds of
// what the CU's vector memory path moved.
//
// LDS: rows of a multiple of 128 bytes, the 16-byte chunks of each group of
// eight XORed with the row's low bits; then rows of scales of a multiple of 16.
constexpr int ROWS_WAVES = 4;
constexpr uint32_t ROWS_LDS = 144 * 1024;         // most that a workgroup's rows and scales may take
struct RowsShape { uint32_t row, sc; };           // bytes per row in LDS
__host__ __device__ __forceinline__ RowsShape rows_shape(int K, bool fp4a) {
  return {((uint32_t)(fp4a ? K / 2 : K) + 127) / 128 * 128, ((uint32_t)K / 32 + 15) / 16 * 16};
}
static uint32_t rows_lds(int M, int K, bool fp4a) {
  const RowsShape s = rows_shape(K, fp4a);
  return (uint32_t)(M < 16 ? M : 16) * (s.row + s.sc) + RPK;           // a row's last piece is read whole
}

struct RowsPiece { u32x4 w[4], ws; };             // five loads
__device__ __forceinline__ void rows_load(RowsPiece& P, const uint8_t* wp, const uint8_t* wsp, int c, int g) {
  P.ws = *reinterpret_cast<const u32x4_a1*>(wsp + c * 16);
#pragma unroll
  for (int s = 0; s < 4; ++s) P.w[s] = ldg16(wp + c * 256 + s * 64 + g * 16);
}
// The piece that K ends in: blocks past K are read from the last block and replaced.
__device__ __forceinline__ void rows_load_tail(RowsPiece& P, const uint8_t* wp, const uint8_t* wsp, int c, int g, int nblk) {
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int b = c * 16 + s * 4 + g, bc = min(b, nblk - 1);
    const u32x4 w = ldg16(wp + bc * 16);
    P.w[s] = b < nblk ? w : u32x4{0, 0, 0, 0};
    P.ws[s] = (b < nblk ? (uint32_t)wsp[bc] : 127u) << (8 * g);
  }
}

struct RowsLds { uint32_t row, sc; int r; };      // this lane's row and scales in LDS, and the row's number
__device__ __forceinline__ RowsLds rows_lane(uint32_t lds, const RowsShape& sh, int rows) {
  const int r = min((int)threadIdx.x & 15, rows - 1);
  return {lds + r * sh.row, lds + rows * sh.row + r * sh.sc, r & 7};
}

template <bool FP4A, bool TAIL>
__device__ __forceinline__ v4f rows_multiply(const RowsPiece& P, const RowsLds& L, v4f acc, int c, int g, int nblk) {
  const u32x4 as = lds_read<u32x4>(L.sc + c * 16);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const v8i w = {(int)P.w[s][0], (int)P.w[s][1], (int)P.w[s][2], (int)P.w[s][3], 0, 0, 0, 0};
    // Chunks of 32 (E2M1) or 16 (E4M3: K = 128 s + 16 g and 64 further) elements; their places in LDS.
    const int i = FP4A ? s * 4 + g : s * 8 + g, past = FP4A ? nblk - c * 16 : 2 * (nblk - c * 16);
    auto chunk = [&](int i) {
      return lds_read<u32x4>(L.row + c * (FP4A ? 256 : 512) + (uint32_t)(i / 8 * 8 + ((i ^ L.r) & 7)) * 16);
    };
    u32x4 lo = chunk(i), hi = {0, 0, 0, 0};
    if (!FP4A) hi = chunk(i + 4);
    uint32_t sa = as[s] >> (8 * g);
    if (TAIL) {                                   // LDS past K holds anything
      if (i >= past) lo = u32x4{0, 0, 0, 0};
      if (i + 4 >= past) hi = u32x4{0, 0, 0, 0};
      if (s * 4 + g >= nblk - c * 16) sa = 127;
    }
    const v8i a = {(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
    const uint32_t sb = P.ws[s] >> (8 * g);
    acc = FP4A ? mfma_fp4_fp4(a, w, acc, sa, sb) : mfma_fp8_fp4(a, w, acc, sa, sb);
  }
  __builtin_amdgcn_sched_barrier(0);
  return acc;
}

// The first RING pieces of a weight row (LONG: it has as many), or all of a shorter one.
template <bool LONG, int RING>
__device__ __forceinline__ void rows_prime(RowsPiece (&P)[RING], const uint8_t* wp, const uint8_t* wsp, int nblk, int g) {
  const int whole = nblk / 16;
  if (LONG) {
#pragma unroll
    for (int r = 0; r < RING; ++r) rows_load(P[r], wp, wsp, r, g);
  } else {
#pragma unroll
    for (int r = 0; r + 1 < RING; ++r)
      if (r < whole) rows_load(P[r], wp, wsp, r, g);
    if (nblk % 16) rows_load_tail(P[RING - 1], wp, wsp, whole, g, nblk);
  }
}
// The tile over all of K, the rows in LDS and the pieces asked for by rows_prime.
template <bool FP4A, bool LONG, int RING>
__device__ __forceinline__ v4f rows_finish(RowsPiece (&P)[RING], const RowsLds& L, const uint8_t* wp, const uint8_t* wsp, int nblk,
                                           int g) {
  const int whole = nblk / 16, tail = nblk % 16;
  v4f acc = {0.f, 0.f, 0.f, 0.f};
  int c = 0;
  if (LONG) {
    for (; c + 2 * RING <= whole; c += RING)
#pragma unroll
      for (int r = 0; r < RING; ++r) {
        acc = rows_multiply<FP4A, false>(P[r], L, acc, c + r, g, nblk);
        rows_load(P[r], wp, wsp, c + RING + r, g);
      }
#pragma unroll
    for (int r = 0; r < RING; ++r) {                                  // the last whole pieces but fewer than RING
      acc = rows_multiply<FP4A, false>(P[r], L, acc, c + r, g, nblk);
      if (c + RING + r < whole) rows_load(P[r], wp, wsp, c + RING + r, g);
    }
    c += RING;
    if (tail) rows_load_tail(P[RING - 1], wp, wsp, whole, g, nblk);
  }
#pragma unroll
  for (int r = 0; r + 1 < RING; ++r)
    if (c + r < whole) acc = rows_multiply<FP4A, false>(P[r], L, acc, c + r, g, nblk);
  if (tail) acc = rows_multiply<FP4A, true>(P[RING - 1], L, acc, whole, g, nblk);
  return acc;
}
// The same where the rows come by DMA that went out before: the loads of LONG rows (five a piece) may be on their way
// while it is waited for.
template <bool FP4A, bool LONG, int RING>
__device__ __forceinline__ v4f rows_run(const RowsLds& L, const uint8_t* wp, const uint8_t* wsp, int nblk, int g) {
  RowsPiece P[RING];
  rows_prime<LONG>(P, wp, wsp, nblk, g);
  __builtin_amdgcn_sched_barrier(0);              // the count is of the loads above
  asm volatile("s_waitcnt vmcnt(%0)" :: "n"(LONG ? RING * 5 : 0) : "memory");
  lds_barrier();
  return rows_finish<FP4A, LONG>(P, L, wp, wsp, nblk, g);
}

// The workgroup's rows (a, a_sc from its first row on) to LDS, and for the first CW wavefronts the 16 x 16 tile of this
// lane's weight row wp, wsp over all of K.  Every wavefront passes one barrier.
template <bool FP4A, int CW>
__device__ __forceinline__ v4f rows_tile(uint32_t lds, const uint8_t* a, const uint8_t* a_sc, int rows, const uint8_t* wp,
                                         const uint8_t* wsp, int K) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, nblk = K / 32, whole = K / RPK;
  const uint32_t rowb = FP4A ? K / 2 : K;
  const RowsShape sh = rows_shape(K, FP4A);
  const uint32_t lsc = lds + rows * sh.row;
  for (int r = wave; r < rows; r += ROWS_WAVES) {
    const uint32_t swz = (lane ^ (r & 7)) * 16;
    for (uint32_t c = 0; c < sh.row; c += 1024)
      if (c + lane * 16 < sh.row) dma16_to_lds(a + (size_t)r * rowb, min(c + swz, rowb - 16), lds + r * sh.row + c);
    if (K % 128 == 0) {
      for (uint32_t c = 0; c < (uint32_t)nblk; c += 256)
        if (c + lane * 4 < (uint32_t)nblk) dma4_to_lds(a_sc + r * nblk, c + lane * 4, lsc + r * sh.sc + c);
    } else {                                      // rows of scales start at any byte
      for (int c = lane; c < nblk; c += 64) lds_write<uint8_t>(lsc + r * sh.sc + c, a_sc[r * nblk + c]);
    }
  }
  const RowsLds L = rows_lane(lds, sh, rows);
  asm volatile("" ::: "memory");
  if (wave >= CW) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    lds_barrier();
    return v4f{0.f, 0.f, 0.f, 0.f};
  }
  if (whole >= 8) return rows_run<FP4A, true, 8>(L, wp, wsp, nblk, g);
  if (whole >= 4) return rows_run<FP4A, true, 4>(L, wp, wsp, nblk, g);
  return rows_run<FP4A, false, 4>(L, wp, wsp, nblk, g);
}

template <bool FP4A, int CW>
__global__ __launch_bounds__(64 * ROWS_WAVES, 2) void fp4_rows_kernel(TileArgs A) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int M = A.M, N = A.N, K = A.K, col = lane & 15, nblk = K / 32;
  const uint32_t nct = (N + 16 * CW - 1) / (16 * CW);
  const int64_t n0 = ((int64_t)(blockIdx.x % nct) * CW + wave) * 16, m0 = (int64_t)(blockIdx.x / nct) * 16;
  const int64_t n = min(n0 + col, (int64_t)N - 1);
  const v4f acc = rows_tile<FP4A, CW>(__builtin_amdgcn_readfirstlane(lds_addr(lds)), A.x + m0 * (FP4A ? K / 2 : K), A.x_sc + m0 * nblk,
                                      (int)min((int64_t)16, M - m0), A.w + n * (K / 2), A.w_sc + n * nblk, K);
  if (wave < CW && n0 + col < N) store_rows(A, acc, m0 + 4 * (lane >> 4), n);
}

// The down product of an FFN of very few rows, from its gate/up values in
// fp32 (h: [M][2 K], gate, then up): every workgroup makes the codes of all
// rows itself, 8 columns a lane, into the same places in LDS, while its
// weights are on their way.  The gate/up product then spreads over all CUs,
// where one that makes the codes has K / 32 workgroups.
template <bool FP4A, int CW>
__global__ __launch_bounds__(64 * ROWS_WAVES, 2) void fp4_down_rows_kernel(TileArgs A, const float* __restrict__ h) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds_[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int M = A.M, N = A.N, K = A.K, g = lane >> 4, nblk = K / 32;
  const int64_t n0 = ((int64_t)blockIdx.x * CW + wave) * 16, n = min(n0 + (lane & 15), (int64_t)N - 1);
  const uint8_t* const wp = A.w + n * (K / 2);
  const uint8_t* const wsp = A.w_sc + n * nblk;
  const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_addr(lds_));
  const RowsShape sh = rows_shape(K, FP4A);
  const uint32_t per_row = K / 8, chunks = M * per_row;
  float gt[8], up[8];
  auto fetch = [&](uint32_t c) {
    const uint32_t t = c / per_row, i = (c - t * per_row) * 8;
    load8(h, false, (int64_t)t * 2 * K + i, gt);
    load8(h, false, (int64_t)t * 2 * K + K + i, up);
  };
  // The wavefronts without columns make the codes; where all have some, all do (their values asked for before the weights,
  // since loads arrive in order).
  constexpr uint32_t MAKERS = 64 * (CW < ROWS_WAVES ? ROWS_WAVES - CW : ROWS_WAVES);
  const uint32_t first = threadIdx.x - (64 * ROWS_WAVES - MAKERS);    // past the end in the others
  if (first < chunks) fetch(first);
  asm volatile("" ::: "memory");
  RowsPiece P[4];
  if (CW == ROWS_WAVES || wave < CW) {
    if (nblk >= 64) rows_prime<true>(P, wp, wsp, nblk, g);
    else rows_prime<false>(P, wp, wsp, nblk, g);
  }
  __builtin_amdgcn_sched_barrier(0);
  for (uint32_t c = first; c < chunks;) {
    uint32_t d[2];
    const uint32_t s = swiglu_codes8<FP4A>(gt, up, d);
    const uint32_t r = c / per_row, i = c - r * per_row;
    const uint32_t at = i * (FP4A ? 4 : 8), chunk = at / 16;          // 16-byte chunks as rows_multiply reads them
    const uint32_t to = lds + r * sh.row + ((chunk & ~7u) | ((chunk ^ r) & 7u)) * 16 + at % 16;
    if (FP4A) lds_write<uint32_t>(to, d[0]);
    else lds_write(to, u32x2{d[0], d[1]});
    if (i % 4 == 0) lds_write<uint8_t>(lds + M * sh.row + r * sh.sc + i / 4, (uint8_t)s);
    c += MAKERS;
    if (c < chunks) fetch(c);
  }
  lds_barrier();
  if (wave >= CW) return;
  const RowsLds L = rows_lane(lds, sh, M);
  const v4f acc = nblk >= 64 ? rows_finish<FP4A, true>(P, L, wp, wsp, nblk, g) : rows_finish<FP4A, false>(P, L, wp, wsp, nblk, g);
  if (n0 + (lane & 15) < N) store_rows(A, acc, 4 * g, n);
}

// Many rows: BM x BN output tiles staged through LDS.  A stage holds K = KS
// (256 with E2M1 activations, 128 with E4M3) of the tile's activation and
// weight rows, brought by LDS DMA NST stages ahead of the matrix cores and
// ordered by vmcnt waits and LDS-only barriers, one barrier per stage.  A
// stage's steps are 32x32x64, the shape in which E2M1 x E2M1 runs at its full
// rate; every step's matrix operations carry the LDS reads of the next step's
// operands between them, across the stage's barrier too.
//
// Rows go to LDS in pieces of 128 bytes where they can: the vector memory
// path takes a lookup per row piece, and with pieces of 64 bytes and a dword
// of scales per row and stage the lookups, not the matrix cores, set the time
// (109 us at 8192 x 4096 x 4096 in E2M1).  For the same reason 16 scale bytes
// of a row (K = 512) go to LDS at a time.
//
// 8192 x 4096 x 4096 takes 75 us in E2M1 (3.7 PFLOP/s) and 106 us in E4M3
// (2.6): the matrix cores are busy for 43 and 62 % of the cycles, the rest
// goes to the first loads and the last stores of each round of tiles and, in
// E2M1, to LDS, whose reads and DMA writes of a stage take as many cycles as
// its matrix operations.
//
// The weights take the instruction's A side and the activations its B side,
// so a lane holds one row of y and four consecutive columns per register
// quad: lane l has row l % 32 and columns 8 q + 4 (l / 32) + [0, 4), q = 0..3.
//
// LDS rows are 64 or 128 bytes in 16-byte chunks; the chunk index is XORed
// with bits of the row so that 8 (and 16) consecutive rows' reads of one
// chunk fall on different banks.  The conflicts that are counted (14 to 19 %
// of the LDS cycles of large tiles) are reads of scales, 16 bytes apart.
typedef float v16f __attribute__((ext_vector_type(16)));

// dma16_to_lds if on is -1, nothing if it is 0 (in a wavefront whose lanes are all active): an instruction that may
// have nothing to do, without a branch around it.
__device__ __forceinline__ void dma16_to_lds_if(int on, const void* base, uint32_t off, uint32_t dst) {
  asm volatile("s_mov_b32 exec_lo, %3\n\ts_mov_b32 exec_hi, %3\n\ts_mov_b32 m0, %2\n\ts_nop 0\n\t"
               "global_load_lds_dwordx4 %0, %1\n\ts_mov_b64 exec, -1"
               :: "v"(off), "s"(base), "s"(__builtin_amdgcn_readfirstlane(dst)), "s"(__builtin_amdgcn_readfirstlane(on)) : "m0");
}

__device__ __forceinline__ int swz4(int r) { return (((r >> 1) ^ (r >> 3)) & 1) | ((r >> 1) & 2); }
__device__ __forceinline__ int swz8(int r) { return (r & 6) | ((r >> 3) & 1); }

__device__ __forceinline__ v8i operand(const u32x4& lo) {
  return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], 0, 0, 0, 0};
}
__device__ __forceinline__ v8i operand(const u32x4& lo, const u32x4& hi) {
  return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// Holds the computation of v before what follows (no instruction).
// ACC: v lives in the accumulation registers, which the compiler uses for
// kernels that LDS limits to one wavefront per SIMD (512 registers each).
template <bool ACC> __device__ __forceinline__ void pin(v16f& v) {
  if (ACC) asm volatile("" : "+a"(v));
  else asm volatile("" : "+v"(v));
}

template <int V> struct Int { static constexpr int value = V; };
template <int N> __device__ __forceinline__ void wait_vm() { asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory"); }

constexpr int XCDS = 8;
constexpr int SCK = 512;                          // K whose scales (16 bytes a row) are fetched at a time

// WM x WN wavefronts of TM x TN 32 x 32 tiles each.  ODD: K % 128 != 0, rows
// of scales start at any byte (where LDS has the room; else such scales go
// through registers, at a wait for all of memory per 512 of K).
template <bool FP4A, bool ODD, int WM, int WN, int TM, int TN, int KS, int NST>
struct TileShape {
  static constexpr int NW = WM * WN, BM = WM * TM * 32, BN = WN * TN * 32;
  static constexpr int RA = FP4A ? KS / 2 : KS, RW = KS / 2;     // bytes of an activation / a weight row per stage
  static constexpr int CA = RA / 16, CW = RW / 16;               // their chunks
  static constexpr int NSC = (BM + BN + 64 * NW - 1) / (64 * NW);     // scale rows per lane (surplus ones repeat the last)
  static constexpr uint32_t OFF_W = BM * RA, STAGE = OFF_W + BN * RW;
  static constexpr uint32_t OFF_S = STAGE * NST, SCALES = NSC * NW * (ODD ? 1280 : 1024), LDS = OFF_S + 2 * SCALES;
  static constexpr int NX = BM * RA / 1024 / NW, NWT = BN * RW / 1024 / NW;   // DMA instructions per wavefront and stage
  static constexpr int NV = NX + NWT;
  static constexpr int SPC = SCK / KS;            // stages per scale chunk
  static constexpr int STEPS = KS / 64;
  static constexpr bool ACC = NW * (160 * 1024 / LDS) < 8;        // fewer than 2 wavefronts per SIMD
  // DMA instructions of stage s + NST that go out in the last step of stage s; the others go out in step 0 of stage s + 1
  static constexpr bool WHOLE = TM * TN <= 2;     // small tiles: whole stages of operands in registers
  static constexpr int FIRST = NST == 2 || WHOLE ? NV : NV / 2;
  static_assert(NX * NW * 1024 == BM * RA && NWT * NW * 1024 == BN * RW, "whole rows");
  static_assert(LDS <= 160 * 1024 && NV * (NST - 1) < 63, "LDS and vmcnt");
};

// SwiGLU + codes of one row's block of 32: gate and up of this lane's 16
// columns 8 q + 4 g + [0, 4); its partner is 32 lanes away.  q, sc: the block's
// codes and scale, written if ok (a block is whole or not there: N % 32 == 0).
template <bool FP4>
__device__ __forceinline__ void tile_codes(const v16f& gate, const v16f& up, int g, bool ok, uint8_t* q, uint8_t* sc) {
  float a[16], amax = 0.0f, gmin = gate[0];
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    a[r] = swiglu_near(gate[r], up[r]);
    amax = near_max(amax, a[r]);
    gmin = fminf(gmin, gate[r]);
  }
  const bool whole = amax == amax;
  amax = fmaxf(amax, __shfl_xor(amax, 32));
  uint32_t s = e8m0_code_for_amax(amax, FP4 ? 2 : 8), d[4];
  const bool sure = whole && gmin > SWIGLU_MIN_G && near_block(amax) && codes_near<FP4, 16>(a, s, d);
  if (!__all(sure || !ok)) {
    amax = 0.0f;
#pragma unroll 1
    for (int h = 0; h < 4; ++h)                                       // four at a time: the double form is long
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (r / 4 == h) {
          a[r] = swiglu(gate[r], up[r]);
          amax = fmaxf(amax, __builtin_fabsf(a[r]));
        }
    amax = fmaxf(amax, __shfl_xor(amax, 32));
    s = e8m0_code_for_amax(amax, FP4 ? 2 : 8);
    codes_scaled<FP4, 16>(a, __builtin_ldexpf(1.0f, 127 - (int)s), d);
  }
  if (FP4) {                                                          // halves: q = 0 | q = 1, q = 2 | q = 3
    const auto x = __builtin_amdgcn_permlane32_swap(d[0], d[1], false, false);
    const uint32_t lo = __builtin_amdgcn_perm(x[1], x[0], 0x05040100), hi = __builtin_amdgcn_perm(x[1], x[0], 0x07060302);
    if (ok) *reinterpret_cast<u32x2*>(q + g * 8) = u32x2{lo, hi};
  } else {
    const auto x = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
    const auto y = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
    if (ok) *reinterpret_cast<u32x4*>(q + g * 16) = u32x4{x[0], x[1], y[0], y[1]};
  }
  if (ok && g == 0) *sc = (uint8_t)s;
}

// What a product leaves: y, or the codes of silu(gate) * up (SWIGLU: a tile
// holds 32 gate columns, then the 32 up columns they meet, and so on).
template <bool FP4A, bool SWIGLU, bool ODD, int WM, int WN, int TM, int TN, int KS, int NST>
__global__ __launch_bounds__(64 * WM * WN, 2) void fp4_tile_kernel(TileArgs A) {
  using S = TileShape<FP4A, ODD, WM, WN, TM, TN, KS, NST>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 31, g = lane >> 5;
  const int wm = wave / WN, wn = wave % WN;
  const int M = A.M, N = A.N, K = A.K;
  const int nblk = K / 32, ns = (K + KS - 1) / KS;
  const int rowx = FP4A ? K / 2 : K, roww = K / 2;

  // XCD-aware order: each XCD takes a run of consecutive tiles, which go down 8 row tiles before the next column tile
  constexpr int CN = SWIGLU ? S::BN / 2 : S::BN;                      // result columns of a tile
  const int nrt = (M + S::BM - 1) / S::BM, nct = (N + CN - 1) / CN;
  const uint32_t tiles = (uint32_t)nrt * nct, per = (tiles + XCDS - 1) / XCDS;   // fewer than 2^24
  const uint32_t t = blockIdx.x % XCDS * per + blockIdx.x / XCDS;
  if (t >= tiles) return;
  const uint32_t grp = t / (8u * nct), in = t - grp * 8u * nct, rows_in = min(8u, nrt - grp * 8u);
  const int rt = __builtin_amdgcn_readfirstlane(grp * 8 + in % rows_in), ct = __builtin_amdgcn_readfirstlane(in / rows_in);
  const int64_t m0 = (int64_t)rt * S::BM, n0 = (int64_t)ct * CN;
  const int mlast = (int)min((int64_t)S::BM, M - m0) - 1, nlast = (int)min((int64_t)CN, N - n0) - 1;   // rows past the end repeat the last one
  // the weight row of the tile's r-th column, from row n0 on
  auto wsrc = [&](int r) {
    return SWIGLU ? (uint32_t)min(r / 64 * 32 + r % 32, nlast) + ((r & 32) ? (uint32_t)N : 0u) : (uint32_t)min(r, nlast);
  };
  const uint8_t* xt = A.x + m0 * rowx;
  const uint8_t* wt = A.w + n0 * roww;

  // this lane's DMA sources: byte offsets from the tile's first row
  uint32_t xoff[S::NX], woff[S::NWT];
  const int c8 = (lane % 8) ^ swz8(wave * 8 + lane / 8), c4 = (lane % 4) ^ swz4(lane / 4);
  auto cx = [&](int i) { return S::CA == 8 ? c8 ^ (S::NW & i & 1) : c4; };   // its chunk of a row piece in instruction i
  auto cw = [&](int i) { return S::CW == 8 ? c8 ^ (S::NW & i & 1) : c4; };   // (an odd NW changes the row's bit 3 with i)
#pragma unroll
  for (int i = 0; i < S::NX; ++i) {
    const int r = (i * S::NW + wave) * (64 / S::CA) + lane / S::CA;
    xoff[i] = (uint32_t)min(r, mlast) * (uint32_t)rowx + cx(i) * 16;
  }
#pragma unroll
  for (int i = 0; i < S::NWT; ++i) {
    const int r = (i * S::NW + wave) * (64 / S::CW) + lane / S::CW;
    woff[i] = wsrc(r) * (uint32_t)roww + cw(i) * 16;
  }
  const uint8_t* srow[S::NSC];                                        // this lane's scale rows: activations, then weights
#pragma unroll
  for (int i = 0; i < S::NSC; ++i) {
    const int r = (i * S::NW + wave) * 64 + lane;
    srow[i] = r < S::BM ? A.x_sc + (m0 + min(r, mlast)) * nblk : A.w_sc + (n0 + wsrc(min(r - S::BM, S::BN - 1))) * nblk;
  }
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(lds));
  const bool ragged = K % KS != 0;                                    // the last stage runs past K: chunks past K
  auto xpast = [&](int i) { return (ns - 1) * KS + cx(i) * (FP4A ? 32 : 16) >= K; };           // read the stage's first
  auto wpast = [&](int i) { return (ns - 1) * KS + cw(i) * 32 >= K; };                         // chunk of their row
  // The i-th DMA instruction of stage s, activations then weights; none of the lanes take part in stages past the last.
  auto issue1 = [&](int s, uint32_t buf, int i) {
    const int on = (s - ns) >> 31;
    if (i < S::NX)
      dma16_to_lds_if(on, xt + (int64_t)s * S::RA, xoff[i < S::NX ? i : 0] - (s == ns - 1 && xpast(i) ? cx(i) * 16 : 0),
                      lds0 + buf + (i * S::NW + wave) * 1024);
    else
      dma16_to_lds_if(on, wt + (int64_t)s * S::RW, woff[i < S::NX ? 0 : i - S::NX] - (s == ns - 1 && wpast(i - S::NX) ? cw(i - S::NX) * 16 : 0),
                      lds0 + buf + S::OFF_W + ((i - S::NX) * S::NW + wave) * 1024);
  };
  // Scales of K = 512 c + [0, 512) of this lane's rows, to the buffer c % 2: by DMA where the 16 bytes are the row's and
  // dword-aligned, else through registers, written to LDS when the chunk is published (put).  Blocks past K get 127;
  // the dword that holds a row's last blocks is read from the row's last four bytes (K >= 128), so no read leaves the
  // row.  Rows start at any byte where K % 128 != 0: with ODD the DMA brings the five dwords that the 16 bytes lie in (the
  // fifth, where they fill four, is the fourth again; a dword with one of the row's bytes in it is readable), the fifth
  // behind the buffer's rows of 16, and a reader shifts by its row's offset.
  u32x4 sreg[S::NSC];
  auto by_dma = [&](int c) { return (ODD || K % 128 == 0) && c * 16 + 16 <= nblk; };
  auto fetch_scales = [&](int c) {
    const int b0 = c * 16;
    if (by_dma(c)) {
#pragma unroll
      for (int i = 0; i < S::NSC; ++i) {
        uint8_t* const to = lds + S::OFF_S + (c & 1) * S::SCALES + (i * S::NW + wave) * 1024;
        const uint32_t o = ODD ? (uint32_t)(uintptr_t)srow[i] & 3 : 0;
        dma16_to_lds(srow[i] - o + b0, to);
        if (ODD) dma4_to_lds(srow[i] - o + b0 + (o ? 16 : 12), lds + S::OFF_S + (c & 1) * S::SCALES + S::NSC * S::NW * 1024 + (i * S::NW + wave) * 256);
      }
    } else {
#pragma unroll
      for (int i = 0; i < S::NSC; ++i)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const int at = min(b0 + 4 * d, nblk - 4), cut = b0 + 4 * d - at;
          const uint32_t v = *reinterpret_cast<const u32_a1*>(srow[i] + at);
          sreg[i][d] = cut == 0 ? v : cut < 4 ? (v >> (8 * cut)) | (0x7F7F7F7Fu << (32 - 8 * cut)) : 0x7F7F7F7Fu;
        }
    }
  };
  auto put_scales = [&](int c) {
    if (by_dma(c)) return;
#pragma unroll
    for (int i = 0; i < S::NSC; ++i)
      lds_write(lds0 + S::OFF_S + (c & 1) * S::SCALES + ((i * S::NW + wave) * 64 + lane) * 16, sreg[i]);
  };

  // Operands of one step; the scale dwords of 256 of K (read from LDS in pairs: dword reads of rows 16 bytes apart meet on
  // a quarter of the banks), and those of the current 128, shifted so that bytes 0 and 2 are the blocks of this lane's
  // half in their two steps.
  struct Regs { u32x4 xlo[TM], xhi[FP4A ? 1 : TM], w[TN]; };
  struct Pairs { u32x2 x[TM], w[TN]; };
  struct Scales { uint32_t x[TM], w[TN]; };
  const uint32_t xrow = (uint32_t)(wm * TM * 32 + lr), wrow = (uint32_t)(wn * TN * 32 + lr);
  const uint32_t xp = xrow * S::RA + (g ^ (S::CA == 8 ? swz8(lr) : swz4(lr))) * 16, wp = S::OFF_W + wrow * S::RW + (g ^ (S::CW == 8 ? swz8(lr) : swz4(lr))) * 16;
  const uint32_t sp = lds0 + S::OFF_S + xrow * 16, sw = lds0 + S::OFF_S + (S::BM + wrow) * 16;
  constexpr int NLD = TN + TM * (FP4A ? 1 : 2), NMM = TM * TN;       // LDS reads and matrix operations of a step
  // LDS addresses of the steps' chunks in the first buffer; a step's chunk is an XOR of bits that the row leaves zero
  uint32_t xa[2 * S::STEPS], wa[S::STEPS];
#pragma unroll
  for (int ks = 0; ks < S::STEPS; ++ks) {
    wa[ks] = (lds0 + wp) ^ (ks * 32);
    xa[2 * ks] = (lds0 + xp) ^ (ks * (FP4A ? 32 : 64));
    xa[2 * ks + 1] = xa[2 * ks] ^ 32;                                 // E4M3: the second half's chunk
  }
  // the it-th LDS read of step ks from the buffer at offset buf (weights first: every matrix operation row needs them)
  auto load1 = [&](Regs& R, uint32_t buf, int ks, int it) {
    if (it < TN) R.w[it] = lds_read<u32x4>(wa[ks] + buf + it * 32 * S::RW);
    else if (FP4A) R.xlo[it - TN] = lds_read<u32x4>(xa[2 * ks] + buf + (it - TN) * 32 * S::RA);
    else {
      const int i = (it - TN) / 2;
      if ((it - TN) % 2 == 0) R.xlo[i] = lds_read<u32x4>(xa[2 * ks] + buf + i * 32 * S::RA);
      else R.xhi[FP4A ? 0 : i] = lds_read<u32x4>(xa[2 * ks + 1] + buf + i * 32 * S::RA);
    }
  };
  Scales off = {};                                                  // ODD: where rows of scales start in their dword
  if (ODD) {
#pragma unroll
    for (int i = 0; i < TM; ++i) off.x[i] = (uint32_t)(uintptr_t)(A.x_sc + (m0 + min((int)xrow + i * 32, mlast)) * nblk) & 3;
#pragma unroll
    for (int i = 0; i < TN; ++i) off.w[i] = (uint32_t)(uintptr_t)(A.w_sc + (n0 + wsrc(wrow + i * 32)) * nblk) & 3;
  }
  const uint32_t fifth = lds0 + S::OFF_S + S::NSC * S::NW * 1024;     // ODD: the fifth dwords
  auto load_pairs = [&](Pairs& H, int k256) {                         // of K = 256 k256 + [0, 256)
    const uint32_t at = ((k256 >> 1) & 1) * S::SCALES, d = (k256 & 1) * 8;
    const bool whole = by_dma(k256 >> 1);
#pragma unroll
    for (int i = 0; i < TM + TN; ++i) {
      const uint32_t row = (i < TM ? sp + i * 32 * 16 : sw + (i - TM) * 32 * 16) + at;
      u32x2 v = lds_read<u32x2>(row + d);
      if (ODD) {
        const uint32_t o = whole ? (i < TM ? off.x[i < TM ? i : 0] : off.w[i < TM ? 0 : i - TM]) : 0;
        const uint32_t n = i < TM ? xrow + i * 32 : S::BM + wrow + (i - TM) * 32;
        const uint32_t next = lds_read<uint32_t>(d ? fifth + at + n * 4 : row + 8);
        v = u32x2{__builtin_amdgcn_alignbyte(v[1], v[0], o), __builtin_amdgcn_alignbyte(next, v[1], o)};
      }
      if (i < TM) H.x[i < TM ? i : 0] = v;
      else H.w[i < TM ? 0 : i - TM] = v;
    }
  };
  auto second = [&](Pairs& H) {
#pragma unroll
    for (int i = 0; i < TM; ++i) H.x[i][0] = H.x[i][1];
#pragma unroll
    for (int i = 0; i < TN; ++i) H.w[i][0] = H.w[i][1];
  };
  auto take = [&](Scales& C, const Pairs& H) {
#pragma unroll
    for (int i = 0; i < TM; ++i) C.x[i] = H.x[i][0] >> (8 * g);
#pragma unroll
    for (int i = 0; i < TN; ++i) C.w[i] = H.w[i][0] >> (8 * g);
  };
  v16f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  auto mma = [&](const Regs& R, const Scales& C, auto half, int q) {  // the q-th matrix operation; half: step % 2
    constexpr int B = 2 * decltype(half)::value;
    const int i = q / TN, j = q % TN;
    const v8i xv = FP4A ? operand(R.xlo[i]) : operand(R.xlo[i], R.xhi[FP4A ? 0 : i]);
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(R.w[j]), xv, acc[i][j], 4, FP4A ? 4 : 0, B,
                                                                (int)C.w[j], B, (int)C.x[i]);
  };
  // One step's matrix operations with the next step's LDS reads and DMA instructions [d0, d1) of stage sd between them:
  // a wavefront stalls at a DMA instruction while the memory path is still taking its last ones, so they come one at a
  // time.  The order is held by scheduling barriers inside a block of code, and by the empty statements at the end (no
  // instruction) beyond it: without them the compiler moves the matrix operations past the next branch, behind the
  // wait for the next stage.
  auto step = [&](const Regs& R, const Scales& C, auto half, Regs& Rn, uint32_t base, int ks, int sd, uint32_t based,
                  int d0, int d1) {
#pragma unroll
    for (int q = 0; q < NMM; ++q) {
#pragma unroll
      for (int it = q * NLD / NMM; it < (q + 1) * NLD / NMM; ++it) load1(Rn, base, ks, it);
      mma(R, C, half, q);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int it = d0 + q * (d1 - d0) / NMM; it < d0 + (q + 1) * (d1 - d0) / NMM; ++it) issue1(sd, based, it);
    }
#pragma unroll
    for (int q = 0; q < NMM; ++q) pin<S::ACC>(acc[q / TN][q % TN]);
  };
  const Int<0> even;
  const Int<1> odd;

  // Zeros in the activations' chunks past K of the last stage, once they have landed (E2M1 weights are finite, so the
  // products are zeros; E4M3 ones may not be).
  auto cut = [&](uint32_t buf) {
#pragma unroll
    for (int i = 0; i < S::NX; ++i)
      if (xpast(i)) lds_write(lds0 + buf + (i * S::NW + wave) * 1024 + lane * 16, u32x4{0, 0, 0, 0});
  };

  // Scale chunks are asked for before the stage that goes out with them, and are needed SPC stages later, when the
  // waits leave NST - 2 later stages in flight at most.
  static_assert(S::SPC >= NST - 2, "a chunk has landed when it is published");
  fetch_scales(0);
  put_scales(0);
  if (K > SCK) fetch_scales(1);
#pragma unroll
  for (int s = 0; s < NST; ++s)
#pragma unroll
    for (int i = 0; i < (s + 1 < NST ? S::NV : S::FIRST); ++i) issue1(s, s * S::STAGE, i);
  if (ns >= NST) wait_vm<S::NV * (NST - 2) + S::FIRST>();             // the first stage and its scales
  else wait_vm<0>();
  if (ragged && ns == 1) cut(0);
  lds_barrier();
  if constexpr (S::WHOLE) {
    // Small tiles: a stage's operands are read from LDS in one go, while the stage before multiplies, so that the LDS
    // latency is met once per stage and not once per step.
    struct Stage { Regs r[S::STEPS]; Scales c[KS / 128]; };
    // The scales of 128 of K: dword d of the buffer at offset at; whole: the buffer was filled by DMA.
    auto load_scales = [&](Scales& C, uint32_t at, int d, bool whole) {
#pragma unroll
      for (int i = 0; i < TM + TN; ++i) {
        const uint32_t row = (i < TM ? sp + i * 32 * 16 : sw + (i - TM) * 32 * 16) + at;
        uint32_t v = lds_read<uint32_t>(row + d * 4);
        if (ODD) {
          const uint32_t o = i < TM ? off.x[i < TM ? i : 0] : off.w[i < TM ? 0 : i - TM];
          const uint32_t n = i < TM ? xrow + i * 32 : S::BM + wrow + (i - TM) * 32;
          const uint32_t next = lds_read<uint32_t>(d < 3 ? row + d * 4 + 4 : fifth + at + n * 4);
          v = __builtin_amdgcn_alignbyte(next, v, whole ? o : 0);
        }
        if (i < TM) C.x[i < TM ? i : 0] = v;
        else C.w[i < TM ? 0 : i - TM] = v;
      }
    };
    auto load_stage = [&](Stage& G, uint32_t buf, int s) {
#pragma unroll
      for (int ks = 0; ks < S::STEPS; ++ks)
#pragma unroll
        for (int it = 0; it < NLD; ++it) load1(G.r[ks], buf, ks, it);
#pragma unroll
      for (int d = 0; d < KS / 128; ++d) {
        const int k128 = s * (KS / 128) + d;
        load_scales(G.c[d], ((k128 >> 2) & 1) * S::SCALES, k128 & 3, by_dma(k128 >> 2));
      }
    };
    auto multiply = [&](Stage& G) {
#pragma unroll
      for (int d = 0; d < KS / 128; ++d) {
#pragma unroll
        for (int i = 0; i < TM; ++i) G.c[d].x[i] >>= 8 * g;
#pragma unroll
        for (int i = 0; i < TN; ++i) G.c[d].w[i] >>= 8 * g;
#pragma unroll
        for (int q = 0; q < NMM; ++q) mma(G.r[2 * d], G.c[d], even, q);
#pragma unroll
        for (int q = 0; q < NMM; ++q) mma(G.r[2 * d + 1], G.c[d], odd, q);
      }
#pragma unroll
      for (int q = 0; q < NMM; ++q) pin<S::ACC>(acc[q / TN][q % TN]);
    };
    Stage G0, G1;
    load_stage(G0, 0, 0);
    int s = 0;
    // A lone wavefront per SIMD is bound by the instructions it issues, so the stages in the middle run without any of
    // the choices below: four stages (the four buffers) at constant LDS offsets, whole scale chunks, whole rows.
    static_assert(NST == 4, "four buffers");
    const uint8_t* xs = xt + (int64_t)NST * S::RA;
    const uint8_t* wst = wt + (int64_t)NST * S::RW;
    auto quick = [&](auto u, Stage& G, Stage& Gn) {                   // stage s with s % 4 == u
      constexpr int U = decltype(u)::value, V = (U + 1) % 4;
      wait_vm<S::NV * (NST - 2)>();
      lds_barrier();
#pragma unroll
      for (int ks = 0; ks < S::STEPS; ++ks)
#pragma unroll
        for (int it = 0; it < NLD; ++it) load1(Gn.r[ks], V * S::STAGE, ks, it);
#pragma unroll
      for (int d = 0; d < KS / 128; ++d) {
        const uint32_t chunk = (FP4A ? (U + 1) >> 1 : (s + U + 1) >> 2) & 1, dword = FP4A ? 2 * ((U + 1) & 1) + d : (U + 1) & 3;
        load_scales(Gn.c[d], chunk * S::SCALES, dword, true);
      }
      if ((U + 1) % S::SPC == 0) fetch_scales((s + U + 1) / S::SPC + 1);   // the next stage starts a chunk
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < S::NX; ++i) dma16_to_lds(xs, xoff[i], lds0 + U * S::STAGE + (i * S::NW + wave) * 1024);
#pragma unroll
      for (int i = 0; i < S::NWT; ++i) dma16_to_lds(wst, woff[i], lds0 + U * S::STAGE + S::OFF_W + (i * S::NW + wave) * 1024);
      xs += S::RA;
      wst += S::RW;
      multiply(G);
    };
    const int last = ns - 1 - (ragged ? 1 : 0);                       // the last stage of whole rows
    for (; s + 3 + NST <= last && by_dma((s + 4) / S::SPC + 1); s += 4) {
      quick(Int<0>{}, G0, G1);
      quick(Int<1>{}, G1, G0);
      quick(Int<2>{}, G0, G1);
      quick(Int<3>{}, G1, G0);
    }
    uint32_t b0 = 0;
    auto stage = [&](int s, Stage& G, Stage& Gn) {
      const uint32_t b1 = b0 + S::STAGE == NST * S::STAGE ? 0 : b0 + S::STAGE;
      const bool chunk = (s + 1) % S::SPC == 0;
      if (chunk) put_scales((s + 1) / S::SPC);
      if (s + NST - 1 < ns) wait_vm<S::NV * (NST - 2)>();
      else wait_vm<0>();
      if (ragged && s + 2 == ns) cut(b1);
      lds_barrier();                                                  // stage s has been read out by every wavefront
      load_stage(Gn, b1, s + 1);
      __builtin_amdgcn_sched_barrier(0);
      if (chunk && ((s + 1) / S::SPC + 1) * SCK < K) fetch_scales((s + 1) / S::SPC + 1);
      if (s + NST < ns) {
#pragma unroll
        for (int i = 0; i < S::NV; ++i) issue1(s + NST, b0, i);
      }
      multiply(G);
      b0 = b1;
    };
    for (; s + 2 < ns; s += 2) {
      stage(s, G0, G1);
      stage(s + 1, G1, G0);
    }
    if (s + 1 < ns) {
      stage(s, G0, G1);
      multiply(G1);
    } else {
      multiply(G0);
    }
  } else {
    Regs R0, R1;
    Pairs H;
    Scales C;
#pragma unroll
    for (int it = 0; it < NLD; ++it) load1(R0, 0, 0, it);
    load_pairs(H, 0);
    take(C, H);
    int s = 0;
    // One scale chunk of stages at a time while there is nothing to choose: whole rows and chunks, every stage that is
    // asked for exists.
    const uint8_t* xs = xt + (int64_t)(NST - 1) * S::RA;              // the stage whose DMA goes out next
    const uint8_t* wst = wt + (int64_t)(NST - 1) * S::RW;
    uint32_t bp = (NST - 1) * S::STAGE, b0 = 0;                       // buffers of stages s - 1 and s
    auto quick_step = [&](const Regs& R, auto half, Regs& Rn, uint32_t buf, int ks, uint32_t bufd, int d0, int d1) {
#pragma unroll
      for (int q = 0; q < NMM; ++q) {
#pragma unroll
        for (int it = q * NLD / NMM; it < (q + 1) * NLD / NMM; ++it) load1(Rn, buf, ks, it);
        mma(R, C, half, q);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int it = d0 + q * (d1 - d0) / NMM; it < d0 + (q + 1) * (d1 - d0) / NMM; ++it)
          if (it < S::NX) dma16_to_lds(xs, xoff[it < S::NX ? it : 0], lds0 + bufd + (it * S::NW + wave) * 1024);
          else dma16_to_lds(wst, woff[it < S::NX ? 0 : it - S::NX], lds0 + bufd + S::OFF_W + ((it - S::NX) * S::NW + wave) * 1024);
      }
#pragma unroll
      for (int q = 0; q < NMM; ++q) pin<S::ACC>(acc[q / TN][q % TN]);
    };
    auto quick = [&](auto u) {                                        // stage s + U
      constexpr int U = decltype(u)::value;
      constexpr bool FIXED = S::SPC % NST == 0;                       // constant buffers
      const uint32_t f0 = FIXED ? U % NST * S::STAGE : b0, fp = FIXED ? (U + NST - 1) % NST * S::STAGE : bp;
      const uint32_t f1 = FIXED ? (U + 1) % NST * S::STAGE : b0 + S::STAGE == NST * S::STAGE ? 0 : b0 + S::STAGE;
      quick_step(R0, even, R1, f0, 1, fp, S::FIRST, S::NV);
      xs += S::RA;
      wst += S::RW;
      if (S::STEPS == 4) {
        second(H);
        quick_step(R1, odd, R0, f0, 2, 0, 0, 0);
        take(C, H);
        quick_step(R0, even, R1, f0, 3, 0, 0, 0);
      }
      wait_vm<S::NV * (NST - 2)>();
      lds_barrier();
      if (U + 1 == S::SPC) fetch_scales((s + U + 1) / S::SPC + 1);
      if (KS == 256) load_pairs(H, s + U + 1);
      else if (U % 2) load_pairs(H, (s + U + 1) / 2);
      else second(H);
      quick_step(R1, odd, R0, f1, 0, f0, 0, S::FIRST);
      take(C, H);
      if (!FIXED) {
        bp = b0;
        b0 = f1;
      }
    };
    const int last = ns - 1 - (ragged ? 1 : 0);                       // the last stage of whole rows
    for (; s + S::SPC - 1 + NST <= last && by_dma(s / S::SPC + 2); s += S::SPC) {
      quick(Int<0>{});
      quick(Int<1>{});
      if constexpr (S::SPC == 4) {
        quick(Int<2>{});
        quick(Int<3>{});
      }
    }
    // steps 0 .. STEPS - 2 of stage s, with what is left of the DMA of stage s - 1 + NST into the buffer of stage s - 1
    auto inner = [&](int s) {
      step(R0, C, even, R1, b0, 1, s - 1 + NST, bp, S::FIRST, S::NV);
      if (S::STEPS == 4) {
        second(H);
        step(R1, C, odd, R0, b0, 2, 0, 0, 0, 0);
        take(C, H);
        step(R0, C, even, R1, b0, 3, 0, 0, 0, 0);
      }
    };
    for (; s + 1 < ns; ++s) {
      const uint32_t b1 = b0 + S::STAGE == NST * S::STAGE ? 0 : b0 + S::STAGE;
      inner(s);
      // the next stage's data is waited for and published; this stage's buffer has been read out by every wavefront
      const bool chunk = (s + 1) % S::SPC == 0;                       // the next stage starts a scale chunk
      if (chunk) put_scales((s + 1) / S::SPC);
      if (NST > 2 && s + NST - 1 < ns) wait_vm<S::NV * (NST - 2)>();  // all but the stages after the next one
      else wait_vm<0>();
      if (ragged && s + 2 == ns) cut(b1);
      lds_barrier();
      if (chunk && ((s + 1) / S::SPC + 1) * SCK < K) fetch_scales((s + 1) / S::SPC + 1);
      if (KS == 256) load_pairs(H, s + 1);
      else if (s % 2) load_pairs(H, (s + 1) / 2);
      else second(H);
      step(R1, C, odd, R0, b1, 0, s + NST, b0, 0, S::FIRST);
      take(C, H);
      bp = b0;
      b0 = b1;
    }
    inner(ns);                                                        // of stage ns - 1; no DMA is left
#pragma unroll
    for (int q = 0; q < NMM; ++q) mma(R1, C, odd, q);
  }

  if constexpr (SWIGLU) {
    // Codes.  A lane and its partner 32 lanes away hold a block of 32 columns of one row, 16 each: four at 8 q + 4 g.
    // Each pair of dwords (or halves) is exchanged so that a lane writes 16 neighbouring columns.
    static_assert(TN % 2 == 0, "gate and up in one wavefront");
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; j += 2) {
        const int64_t m = m0 + wm * TM * 32 + i * 32 + lr, n = n0 + wn * TN * 16 + j * 16;
        if (A.fp4mid) tile_codes<true>(acc[i][j], acc[i][j + 1], g, m < M && n < N, A.q + m * (N / 2) + n / 2, A.q_sc + m * (N / 32) + n / 32);
        else tile_codes<false>(acc[i][j], acc[i][j + 1], g, m < M && n < N, A.q + m * N + n, A.q_sc + m * (N / 32) + n / 32);
      }
    return;
  }
  // Results.  Each wavefront turns 32 rows at a time in its own part of LDS, so that a store instruction writes whole
  // runs of a row: 16 bytes a lane, at whatever alignment the row has (2 bytes where N is odd), the row's last piece by
  // elements.
  uint8_t* const y = static_cast<uint8_t*>(A.y);
  constexpr int WC = TN * 32;                                         // columns of a wavefront
  constexpr uint32_t PITCH = WC * 4 + 16;                             // + 16: rows start on different banks
  static_assert(S::NW * 32 * PITCH <= S::OFF_S, "epilogue LDS");
  lds_barrier();                                                      // every wavefront has read its operands
  const uint32_t mine = lds0 + wave * 32 * PITCH;
  const int nw = (int)min((int64_t)WC, N - n0 - wn * WC);             // this wavefront's columns
  auto store = [&](auto esize) {                                      // bytes of a result
    constexpr int ESZ = decltype(esize)::value, LPR = WC * ESZ / 16, PER = 16 / ESZ;   // lanes per row, elements per lane
    constexpr int RPP = 64 / LPR, PASSES = 32 / RPP, GROUP = PASSES < 4 ? PASSES : 4;  // rows at a time; LDS reads in flight
    const int r0 = lane / LPR, c0 = lane % LPR * PER;
    const uint32_t from = mine + r0 * PITCH + c0 * ESZ;
    const int64_t step = (int64_t)RPP * N * ESZ;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const v16f& c = acc[i][j];
          const uint32_t at = mine + lr * PITCH + (j * 32 + 8 * q + 4 * g) * ESZ;
          if (ESZ == 2) lds_write(at, u32x2{bf16_pair(c[4 * q], c[4 * q + 1]), bf16_pair(c[4 * q + 2], c[4 * q + 3])});
          else
            lds_write(at, u32x4{__float_as_uint(c[4 * q]), __float_as_uint(c[4 * q + 1]), __float_as_uint(c[4 * q + 2]),
                                __float_as_uint(c[4 * q + 3])});
        }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");              // the wavefront's own writes
      const int64_t mb = m0 + wm * TM * 32 + i * 32;
      const int64_t left = M - mb;                                    // rows
      uint8_t* to = y + ((mb + r0) * N + n0 + wn * WC + c0) * ESZ;
#pragma unroll
      for (int p0 = 0; p0 < PASSES; p0 += GROUP) {
        u32x4 d[GROUP];
#pragma unroll
        for (int p = 0; p < GROUP; ++p) d[p] = lds_read<u32x4>(from + (p0 + p) * RPP * PITCH);
#pragma unroll
        for (int p = 0; p < GROUP; ++p, to += step) {
          if (left >= 32 && nw == WC) {
            *reinterpret_cast<u32x4_a1*>(to) = d[p];
            continue;
          }
          if (r0 + (p0 + p) * RPP >= left) continue;
          if (c0 + PER <= nw) *reinterpret_cast<u32x4_a1*>(to) = d[p];
          else
#pragma unroll
            for (int e = 0; e < PER; ++e) {
              if (c0 + e >= nw) continue;
              if (ESZ == 2) reinterpret_cast<uint16_t*>(to)[e] = (uint16_t)(d[p][e / (4 / ESZ)] >> (16 * (e % 2)));
              else reinterpret_cast<uint32_t*>(to)[e] = d[p][e / (4 / ESZ)];
            }
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
  };
  if (A.bf16_out) store(Int<2>{});
  else store(Int<4>{});
}

template <bool FP4A, bool SWIGLU, bool ODD, int WM, int WN, int TM, int TN, int KS, int NST>
static void launch_tile_of(const TileArgs& a, hipStream_t stream) {
  using S = TileShape<FP4A, ODD, WM, WN, TM, TN, KS, NST>;
  constexpr int CN = SWIGLU ? S::BN / 2 : S::BN;
  const int64_t tiles = (int64_t)((a.M + S::BM - 1) / S::BM) * ((a.N + CN - 1) / CN);
  const dim3 grid((unsigned)((tiles + XCDS - 1) / XCDS * XCDS)), block(64 * S::NW);
  hipLaunchKernelGGL((fp4_tile_kernel<FP4A, SWIGLU, ODD, WM, WN, TM, TN, KS, NST>), grid, block, 0, stream, a);
}
template <bool FP4A, bool SWIGLU, int WM, int WN, int TM, int TN, int KS, int NST>
static void launch_tile(const TileArgs& a, hipStream_t stream) {
  using S = TileShape<FP4A, false, WM, WN, TM, TN, KS, NST>;
  constexpr uint32_t CU = 160 * 1024;             // ODD where it leaves as many workgroups per CU
  if constexpr (CU / (S::LDS + 2 * S::NSC * S::NW * 256) == CU / S::LDS) {
    if (a.K % 128 != 0) return launch_tile_of<FP4A, SWIGLU, true, WM, WN, TM, TN, KS, NST>(a, stream);
  }
  launch_tile_of<FP4A, SWIGLU, false, WM, WN, TM, TN, KS, NST>(a, stream);
}

static int64_t tiles_of(int M, int N, int bm, int bn) { return ((int64_t)M + bm - 1) / bm * (((int64_t)N + bn - 1) / bn); }
template <bool FP4A, int CW> static void launch_rows_of(const TileArgs& t, hipStream_t stream) {
  const dim3 grid((unsigned)(tiles_of(t.M, t.N, 16, 16 * CW)));       // CW = 4 past 512: fewer than 2^24
  hipLaunchKernelGGL((fp4_rows_kernel<FP4A, CW>), grid, dim3(64 * ROWS_WAVES), rows_lds(t.M, t.K, FP4A), stream, t);
}
// Up to 16 rows by a wavefront alone: n wavefronts of 16 columns, at most one per CU and short rows; more of them where the
// rows are very short, since what LDS saves grows with both; and rows that LDS does not hold, against tiles.  Alone / through
// LDS (tiles where marked t) at M = 1 and 16, us, weights from memory:
//   E2M1 4096 x 576 2.6 / 3.2, 2.9 / 4.2; 4096 x 4096 3.8 / 4.3, 4.7 / 5.3; 4096 x 8192 7.3 / 7.2, 8.3 / 8.0;
//        8192 x 576 3.1 / 3.7, 3.3 / 4.5; 8192 x 1536 3.5 / 3.9, 4.0 / 5.0; 16384 x 576 3.5 / 4.1, 3.8 / 5.0;
//        16384 x 1536 5.2 / 5.5, 5.8 / 6.3; 16384 x 4096 9.7 / 9.6, 12.3 / 10.6
//   E4M3 4096 x 2048 3.3 / 3.5, 3.8 / 4.6; 4096 x 4096 4.7 / 4.5, 5.8 / 5.8; 4096 x 8192 8.9 / 7.0, 10.3 / 8.9;
//        8192 x 576 3.3 / 3.7, 3.6 / 4.6; 8192 x 1536 3.6 / 3.8, 4.4 / 5.1; 16384 x 576 3.7 / 4.0, 4.4 / 5.1;
//        16384 x 1536 5.2 / 5.3, 6.9 / 6.6; 16384 x 4096 10.5 / 9.9, 15.7 / 11.2
//        32768 x 256 4.6 / 4.2, 6.2 / 5.3; M = 16: 4096 x 10240 12.9 / t 21.1, 4096 x 16384 18.7 / t 29.9, 8192 x 16384 27.5 / t 29.7,
//        12288 x 16384 39.2 / t 23.8
static bool alone(int M, int64_t n, int K, bool fp4a) {
  if (M > 16) return false;
  if (rows_lds(M, K, fp4a) > ROWS_LDS) return n <= 512;
  return (n <= 256 && (fp4a ? K / 2 : K) <= 2048) || (n <= 1024 && K <= 1536 && n * K <= 1 << 20);
}
template <bool FP4A> static const char* launch_rows(const TileArgs& t, hipStream_t stream) {
  const int64_t n = tiles_of(t.M, t.N, 16, 16);
  if (alone(t.M, n, t.K, FP4A)) {
    hipLaunchKernelGGL((fp4_lone_kernel<FP4A, 1>), dim3((unsigned)n), dim3(64), 0, stream, t);
    return FP4A ? "fp4:lone16_a4" : "fp4:lone16_a8";
  }
  // K < 128, more than 16 rows (in fewer than 2^32 threads).  So / through LDS, us, E2M1 and E4M3: 17 x 1024 x 96 2.8 / 3.8,
  // 2.9 / 3.9; 256 x 8192 x 96 9.3 / 13.1, 10.2 / 13.3; 4096 x 8192 x 96 111 / 199, 127 / 204; 4096 x 1024 x 32 16.5 / 24.9, 18.5 / 25.5
  const int64_t n64 = tiles_of(t.M, t.N, 64, 16);
  if (t.K < 128 && t.M > 16 && n64 < 1 << 24) {
    hipLaunchKernelGGL((fp4_lone_kernel<FP4A, 4>), dim3((unsigned)n64), dim3(256), 0, stream, t);
    return FP4A ? "fp4:lone64_a4" : "fp4:lone64_a8";
  }
  if (n <= 256) launch_rows_of<FP4A, 1>(t, stream);
  else if (n <= 512) launch_rows_of<FP4A, 2>(t, stream);
  else launch_rows_of<FP4A, 4>(t, stream);
  return FP4A ? "fp4:rows16_a4" : "fp4:rows16_a8";
}

// Which kernel runs (M, N, K), by how many workgroups each shape gives.  Times at N = K = 4096, E2M1 / E4M3 activations:
//   rows (16 at a time, 512 wavefronts):  M = 1 4.2 / 4.5 us, 16 4.8 / 6.0, 32 6.3 / 6.9, 48 8.5 / 9.2; N = 1024: M = 64
//                                         5.1 / 5.8 (32 x 64: 6.3 / 8.0), 128 6.0 / 6.8 (6.3 / 8.0)
//   32 x 64 (2 wavefronts):               M = 32 6.5 / 8.3, 48 6.4 / 8.3, 128 7.0 / 8.8, 256 9.3 / 11.8
//   64 x 64 (4, two workgroups per CU):   M = 48 7.4 / 9.2, 256 7.9 / 10.0, 512 10.6 / 15.2, 1024 20.3 / 26.9
//   128 x 128 (4, two per CU):            M = 256 14.4 / 17.1, 512 13.0 / 17.8, 1024 16.6 / 20.8
//   128 x 256 (8, one per CU):            M = 1024 20.0 / 26.5, 1500 21.9 / 28.5 (128 x 128: 23.7 / 32.1), 2048 24.7 / 34.2
//                                         (26.6 / 37.2), 4096 46.8 / 66.8
//   256 x 256 (8, one per CU):            M = 4096 38.6 / 56.2, about 1.6 times a full round of 128 x 128
enum class Fp4Kernel { rows, t32x64, t64x64, t128x128, t128x256, t256x256 };
// Past 512 tiles of 64 x 64.
static Fp4Kernel pick_large(int M, int N) {
  const int64_t t128 = tiles_of(M, N, 128, 128), t256 = tiles_of(M, N, 256, 256);
  if (t128 > 256 && tiles_of(M, N, 128, 256) <= 256) return Fp4Kernel::t128x256;
  return (t256 + 255) / 256 * 8 <= (t128 + 511) / 512 * 5 ? Fp4Kernel::t256x256 : Fp4Kernel::t128x128;
}
static Fp4Kernel pick_kernel(int M, int N, int K, bool fp4a) {
  const int64_t n = tiles_of(M, N, 16, 16);
  if (((M <= 16 || n <= 512) && rows_lds(M, K, fp4a) <= ROWS_LDS) || alone(M, n, K, fp4a)) return Fp4Kernel::rows;
  if (K < 128) return Fp4Kernel::rows;                                // the tiles' scale reads need four blocks a row
  if (tiles_of(M, N, 32, 64) <= 256) return Fp4Kernel::t32x64;        // one per CU
  if (tiles_of(M, N, 64, 64) <= 512) return Fp4Kernel::t64x64;        // two per CU
  return pick_large(M, N);
}

template <bool FP4A>
static const char* launch_product(const TileArgs& t, hipStream_t stream) {
  switch (pick_kernel(t.M, t.N, t.K, FP4A)) {
    case Fp4Kernel::t32x64:
      launch_tile<FP4A, false, 1, 2, 1, 1, FP4A ? 256 : 128, 4>(t, stream);
      return FP4A ? "fp4:tile32x64_a4" : "fp4:tile32x64_a8";
    case Fp4Kernel::t64x64:
      launch_tile<FP4A, false, 2, 2, 1, 1, FP4A ? 256 : 128, 4>(t, stream);
      return FP4A ? "fp4:tile64x64_a4" : "fp4:tile64x64_a8";
    case Fp4Kernel::t128x128:
      launch_tile<FP4A, false, 2, 2, 2, 2, FP4A ? 256 : 128, FP4A ? 2 : 3>(t, stream);
      return FP4A ? "fp4:tile128x128_a4" : "fp4:tile128x128_a8";
    case Fp4Kernel::t128x256:
      launch_tile<FP4A, false, 2, 4, 2, 2, FP4A ? 256 : 128, FP4A ? 2 : 3>(t, stream);
      return FP4A ? "fp4:tile128x256_a4" : "fp4:tile128x256_a8";
    case Fp4Kernel::t256x256:
      launch_tile<FP4A, false, FP4A ? 2 : 4, FP4A ? 4 : 2, FP4A ? 4 : 2, FP4A ? 2 : 4, FP4A ? 256 : 128, FP4A ? 2 : 3>(t, stream);
      return FP4A ? "fp4:tile256x256_a4" : "fp4:tile256x256_a8";
    default: break;
  }
  return launch_rows<FP4A>(t, stream);
}

hipError_t launch_fp4_gemm(const uint8_t* a, const uint8_t* a_sc, bool fp4a, const uint8_t* w, const uint8_t* w_sc,
                           int M, int N, int K, void* y, bool bf16_out, hipStream_t stream, const char** variant) {
  const TileArgs t{a, a_sc, w, w_sc, M, N, K, y, bf16_out, nullptr, nullptr, false};
  *variant = fp4a ? launch_product<true>(t, stream) : launch_product<false>(t, stream);
  return hipGetLastError();
}

static size_t a256(size_t b) { return (b + 255) / 256 * 256; }

// Gate/up of few rows: one workgroup per 16 rows and block of 32 intermediate
// columns; its four wavefronts take 16 gate or 16 up columns each, meet in
// LDS, and 16 lanes per row make the block's codes, two neighbouring columns
// a lane.  16 rows at H = 4096, I = 2048 take about 8.5 (E2M1) and 9.5 us: 64
// workgroups are all there is to spread, and a CU reads its 136 KB of weights
// in about 4 us.
template <bool FP4A>
__global__ __launch_bounds__(256, 2) void fp4_gate_up_rows_kernel(TileArgs A) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  __shared__ float h[16][4][17];                  // [row][gate, gate, up, up][column]; rows apart by 68: few conflicts
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = lane & 15, g = lane >> 4;
  const int I = A.N, K = A.K, nblk = K / 32;
  const uint32_t nb = I / 32;
  const int64_t n0 = (int64_t)(blockIdx.x % nb) * 32, m0 = (int64_t)(blockIdx.x / nb) * 16;
  const int64_t n = n0 + (wave & 1) * 16 + col + (wave >= 2 ? I : 0);
  const v4f acc = rows_tile<FP4A, 4>(__builtin_amdgcn_readfirstlane(lds_addr(lds)), A.x + m0 * (FP4A ? K / 2 : K), A.x_sc + m0 * nblk,
                                     (int)min((int64_t)16, A.M - m0), A.w + n * (K / 2), A.w_sc + n * nblk, K);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[4 * g + i][wave][col] = acc[i];
  __syncthreads();
  const int row = threadIdx.x >> 4, c = (threadIdx.x & 15) * 2;       // a DPP row of 16 lanes holds one block
  const int64_t r = m0 + row;
  const float g0 = h[row][c >> 4][c & 15], g1 = h[row][c >> 4][(c & 15) + 1];
  const float u0 = h[row][2 + (c >> 4)][c & 15], u1 = h[row][2 + (c >> 4)][(c & 15) + 1];
  float a0 = swiglu_near(g0, u0), a1 = swiglu_near(g1, u1);
  float amax = near_max(__builtin_fabsf(a0), a1);
  const bool whole = amax == amax;
  amax = row16_max(amax);
  const int emax = A.fp4mid ? 2 : 8;
  uint32_t s = e8m0_code_for_amax(amax, emax), d;
  auto codes = [&](float f) -> uint32_t {
    if (A.fp4mid) return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, a0 * f, a1 * f, 1.0f, 0) & 0xFFu;
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(__builtin_amdgcn_fmed3f(a0 * f, -448.0f, 448.0f),
                                                     __builtin_amdgcn_fmed3f(a1 * f, -448.0f, 448.0f), 0, false) & 0xFFFFu;
  };
  const float f = __builtin_ldexpf(1.0f, 127 - (int)s);
  d = codes(f * (1.0f - SWIGLU_EPS));
  const bool sure = whole && fminf(g0, g1) > SWIGLU_MIN_G && near_block(amax) && d == codes(f * (1.0f + SWIGLU_EPS));
  if (!__all(sure)) {
    a0 = swiglu(g0, u0);
    a1 = swiglu(g1, u1);
    s = e8m0_code_for_amax(row16_max(fmaxf(__builtin_fabsf(a0), __builtin_fabsf(a1))), emax);
    d = codes(__builtin_ldexpf(1.0f, 127 - (int)s));
  }
  if (r >= A.M) return;
  if (A.fp4mid) A.q[r * (I / 2) + (n0 + c) / 2] = (uint8_t)d;
  else *reinterpret_cast<uint16_t*>(A.q + r * I + n0 + c) = (uint16_t)d;
  if (c == 0) A.q_sc[r * nb + n0 / 32] = (uint8_t)s;
}

// The kernel by the same counts as pick_kernel, of tiles that hold both halves of a block in one wavefront.  The whole FFN
// at H = 4096, E2M1 / E4M3, us:
//   rows (one workgroup per CU):          48 rows, I = 2048 14.1 / 15.9, 64 14.1 / 16.1, 96 18.4 / 20.4; 128, I = 576 13.7 / 14.5
//   64 x 64 (2 wavefronts, one per CU):   48 rows, I = 2048 13.8 / 18.6, 64 14.6 / 18.9, 96 14.4 / 19.6; 128, I = 576 14.1 / 17.7
//   64 x 128:                             48 rows, I = 2048 16.6 / 20.5, 256 18.2 / 22.1 (64 x 64: 16.2 / 21.2)
//   128 x 256, one round:                 512 rows, I = 8192 46.1 / 66.6 (128 x 128: 47.1 / 68.6)
template <bool FP4A>
static const char* launch_gate_up(const TileArgs& t, hipStream_t stream) {
  const int M = t.M, N = 2 * t.N;
  constexpr int KS = FP4A ? 256 : 128, NB = FP4A ? 2 : 3;
  const int64_t rows = (int64_t)(t.N / 32) * ((M + 15) / 16);
  if (((M <= 16 || rows <= 256) && rows_lds(M, t.K, FP4A) <= ROWS_LDS) || t.K < 128) {
    const dim3 grid((unsigned)rows);
    hipLaunchKernelGGL(fp4_gate_up_rows_kernel<FP4A>, grid, dim3(64 * ROWS_WAVES), rows_lds(M, t.K, FP4A), stream, t);
    return "fp4_ffn:rows16+";
  }
  if (tiles_of(M, N, 64, 64) <= 256) {
    launch_tile<FP4A, true, 2, 1, 1, 2, KS, 4>(t, stream);
    return "fp4_ffn:tile64x64+";
  }
  if (tiles_of(M, N, 64, 128) <= 256) {
    launch_tile<FP4A, true, 2, 2, 1, 2, KS, 4>(t, stream);
    return "fp4_ffn:tile64x128+";
  }
  switch (pick_large(M, N)) {
    case Fp4Kernel::t128x256:
      launch_tile<FP4A, true, 2, 4, 2, 2, KS, NB>(t, stream);
      return "fp4_ffn:tile128x256+";
    case Fp4Kernel::t256x256:
      launch_tile<FP4A, true, FP4A ? 2 : 4, FP4A ? 4 : 2, FP4A ? 4 : 2, FP4A ? 2 : 4, KS, NB>(t, stream);
      return "fp4_ffn:tile256x256+";
    default: break;
  }
  launch_tile<FP4A, true, 2, 2, 2, 2, KS, NB>(t, stream);
  return "fp4_ffn:tile128x128+";
}

// [codes of the intermediate][its scales]
// Up to this many rows the gate/up values go to the down product in fp32: what the codes cost every workgroup grows with
// T I, what spreading the gate/up product over all CUs saves with H.  The FFN in E2M1 / E4M3, us, weights from memory, so and
// with the codes made by the gate/up product (the border's last rows in, first out):
//   H = 512:   I = 96, 16 rows 4.9 / 5.2, 6.4 / 6.5; I = 576, 2 rows 4.9 / 5.1, 5.5 / 5.6, 3 rows 5.9 / 6.0, 5.6 / 5.9
//   H = 1024:  I = 576, 4 rows 6.4 / 6.7, 6.7 / 7.0; I = 1056, 2 rows 6.5 / 6.8, 6.7 / 6.9, 3 rows 7.4 / 7.8, 6.9 / 7.1
//   H = 2048:  I = 576, 4 rows 7.0 / 7.5, 7.7 / 8.0, 8 rows 7.9 / 8.3, 8.0 / 8.2; I = 2048, 1 row 7.2 / 7.9, 7.9 / 8.3, 2 rows
//              8.2 / 8.9, 8.1 / 8.4
//   H = 4096:  I = 576, 1 row 6.4 / 7.2, 9.7 / 10.2, 8 rows 8.8 / 9.8, 10.4 / 11.2, 16 rows 11.6 / 13.0, 11.1 / 12.0;
//              I = 2048, 1 row 8.7 / 9.2, 10.7 / 11.7, 2 rows 9.8 / 10.3, 11.0 / 11.6, 4 rows 12.3 / 13.1, 11.4 / 12.1;
//              I = 4096, 1 row 12.5 / 13.1, 12.8 / 13.5
//   H = 8192:  I = 576, 16 rows 14.1 / 15.3, 18.9 / 19.8; I = 1056, 8 rows 14.4 / 15.2, 17.8 / 18.6; I = 2048, 4 rows
//              14.7 / 15.3, 17.3 / 17.8, 8 rows 18.0 / 19.1, 17.9 / 18.7; I = 4096, 1 row 20.7 / 21.0, 20.0 / 20.3, 2 rows
//              22.3 / 22.9, 20.6 / 21.4
//   H = 16384: I = 2048, 8 rows 22.4 / 23.7, 29.2 / 30.2; I = 4096, 4 rows 35.4 / 36.2, 35.7 / 37.1
// Between I = 2048 and 4096 the product has more than 256 column tiles and less is saved.  Past it they are more than 512,
// which launch_rows takes four to a workgroup: half of the CUs idle, 2 to 7 us lost (H = 8192, 1 row: I = 4608 25.5 / 25.6
// against 20.9 / 21.3, I = 8192 35.9 / 36.2 against 30.1 / 30.4).
static int ffn_h_rows(int H, int I) {
  if (I > 4096) return 0;
  const int rows = (I > 2048 ? H : H + H / 4 + 1024) / I;
  return rows < 16 ? rows : 16;
}

// Enough for fewer rows too.
size_t fp4_ffn_ws_bytes(int T, int H, int I, bool fp4mid) {
  const size_t codes = a256((size_t)T * (fp4mid ? I / 2 : I)) + a256((size_t)T * (I / 32));
  const int rows = T < ffn_h_rows(H, I) ? T : ffn_h_rows(H, I);
  const size_t h = a256((size_t)rows * 2 * I * 4);
  return codes > h ? codes : h;
}

template <bool FP4A> static void launch_down_rows(const TileArgs& t, const float* h, hipStream_t stream) {
  const uint32_t lds = rows_lds(t.M, t.K, FP4A);
  const int64_t n = tiles_of(t.M, t.N, 16, 16);
  if (n <= 256) hipLaunchKernelGGL((fp4_down_rows_kernel<FP4A, 1>), dim3((unsigned)n), dim3(64 * ROWS_WAVES), lds, stream, t, h);
  else hipLaunchKernelGGL((fp4_down_rows_kernel<FP4A, 4>), dim3((unsigned)((t.N + 63) / 64)), dim3(64 * ROWS_WAVES), lds, stream, t, h);
}

hipError_t launch_fp4_ffn(const uint8_t* x, const uint8_t* x_sc, bool fp4x, int T, int H, const uint8_t* w13,
                          const uint8_t* w13_sc, const uint8_t* w2, const uint8_t* w2_sc, int I, bool fp4mid, void* y,
                          bool bf16_out, void* ws, hipStream_t stream, const char** variant) {
  if (T <= ffn_h_rows(H, I)) {
    float* const h = static_cast<float*>(ws);
    const hipError_t e = launch_fp4_gemm(x, x_sc, fp4x, w13, w13_sc, T, 2 * I, H, h, false, stream, variant);
    if (e != hipSuccess) return e;
    const TileArgs t{nullptr, nullptr, w2, w2_sc, T, H, I, y, bf16_out, nullptr, nullptr, false};
    if (fp4mid) launch_down_rows<true>(t, h, stream);
    else launch_down_rows<false>(t, h, stream);
    *variant = "fp4_ffn:h+";
    return hipGetLastError();
  }
  uint8_t* q = static_cast<uint8_t*>(ws);
  uint8_t* q_sc = q + a256((size_t)T * (fp4mid ? I / 2 : I));
  const TileArgs t{x, x_sc, w13, w13_sc, T, I, H, nullptr, false, q, q_sc, fp4mid};
  const char* v = fp4x ? launch_gate_up<true>(t, stream) : launch_gate_up<false>(t, stream);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  e = launch_fp4_gemm(q, q_sc, fp4mid, w2, w2_sc, T, H, I, y, bf16_out, stream, variant);
  *variant = v;
  return e;
}

}  // namespace mx
