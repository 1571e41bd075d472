// Products of E4M3 codes with an fp32 scale for each block of 128 along the
// reduction:
//   y[m][n] = sum_b (sa[m][b] * sw[n'][b]) * P_b[m][n],  P_b = sum over block b of a[m][k] * w[n][k]
// with n' = n / 128 (weights in 128 x 128 tiles) or n (both operands by rows:
// the gradient of weights).  One matrix, the experts' matrices over rows that
// are sorted by expert, and the experts' weight gradients over blocks of K
// that are.
//
// Canonical order: P_b is one 16x16x128 step of the matrix cores from zero, the
// two scales are multiplied in fp32, and acc = fma(P_b, scale, acc) over the
// blocks in order.  Every kernel keeps to it, so a row's bits do not depend on
// M, on the other rows or on the kernel.  A block that K ends in is filled up
// with zeros.
#include "b128_launch.hpp"
#include "group_device.hpp"
#include "lds_device.hpp"
#include "mx_cast.hpp"

namespace mx {

// W (A side: 16 rows n) x X (B side: 16 rows m), K = 128, from zero: lane l holds row m = l % 16 and columns
// n = 4 (l / 16) + [0, 4).
__device__ __forceinline__ v4f block_product(const v8i& w, const v8i& x) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ v8i operand8(const u32x4& lo, const u32x4& hi) {
  return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// What a workgroup works on: a matrix of nrows x ncols results over blocks [0, nkb).
struct B128Task {
  const uint8_t* x; const float* x_sc; const uint8_t* w; const float* w_sc;
  int rows, cols, nkb, K;                         // K: elements in the blocks (a multiple of 16)
  int64_t y0;                                     // first result
};

// ---------------------------------------------------------------------------
// Few rows: a workgroup per 16 columns and 16 MT rows.  Its four wavefronts
// take every fourth block of K, both operands straight to registers, and leave
// each block's products in LDS; then a thread per result adds them up in order.
constexpr int ROWS_CHUNK = 64;                    // 16 x 16 products held in LDS at a time

template <int MT, bool WROWS, B128Mode MODE>
__global__ __launch_bounds__(256, 2) void b128_rows_kernel(B128Args A) {
  constexpr int CH = ROWS_CHUNK / MT;             // blocks of K per chunk
  constexpr int RING = MT == 1 ? 8 : MT == 2 ? 4 : 2;
  static_assert(CH / 4 >= RING, "a wavefront's ring is at most its blocks of a chunk");
  __shared__ __attribute__((aligned(1024))) float prod[CH][MT][16][16];
  __shared__ float sa[CH][MT * 16], sw[CH][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const uint32_t nct = (uint32_t)(((int64_t)A.N + 15) / 16), rt = blockIdx.x / nct;
  const int n0 = (int)(blockIdx.x - rt * nct) * 16;
  const int nkb = (A.K - 1) / 128 + 1;
  int64_t m0 = (int64_t)rt * 16 * MT;
  int rows = (int)min((int64_t)16 * MT, A.M - m0);
  const uint8_t* w = A.w;
  const float* w_sc = A.w_sc;
  if (MODE == B128Mode::grouped) {
    const GroupTile t = find_tile(A.offsets, A.E, A.M, 16 * MT, rt);
    if (t.e < 0) return;
    m0 = t.row0 + (int64_t)t.tile * 16 * MT;
    rows = min(16 * MT, t.rows - t.tile * 16 * MT);
    w += (int64_t)t.e * A.N * A.K;
    w_sc += (int64_t)t.e * ((A.N - 1) / 128 + 1) * nkb;
  }
  const int64_t n = min(n0 + col, A.N - 1);       // columns past the last repeat it, as rows do; they are not stored
  const uint8_t* const wp = w + n * A.ld;
  const uint8_t* xp[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) xp[i] = A.a + (m0 + min(i * 16 + col, rows - 1)) * A.ld;

  struct Piece { u32x4 wlo, whi, xlo[MT], xhi[MT]; };
  auto load = [&](Piece& P, int b) {
    const int k = b * 128 + g * 16, k0 = min(k, A.K - 16), k1 = min(k + 64, A.K - 16);   // past K: the row's last 16 again
    P.wlo = ldg16(wp + k0);
    P.whi = ldg16(wp + k1);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      P.xlo[i] = ldg16(xp[i] + k0);
      P.xhi[i] = ldg16(xp[i] + k1);
    }
  };
  auto multiply = [&](const Piece& P, int b, int at) {
    const int k = b * 128 + g * 16;
    const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const v4f p = block_product(operand8(P.wlo, P.whi),
                                  operand8(k < A.K ? P.xlo[i] : zero, k + 64 < A.K ? P.xhi[i] : zero));
      *reinterpret_cast<v4f*>(&prod[at][i][col][4 * g]) = p;
    }
  };
  Piece R[RING];
#pragma unroll
  for (int r = 0; r < RING; ++r)
    if (wave + 4 * r < nkb) load(R[r], wave + 4 * r);

  float acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = 0.0f;
  for (int b0 = 0; b0 < nkb; b0 += CH) {
    const int nb = min(CH, nkb - b0);
    for (int e = threadIdx.x; e < nb * 16 * MT; e += 256) {
      const int b = e / (16 * MT), m = e % (16 * MT);
      sa[b][m] = A.a_sc[(m0 + min(m, rows - 1)) * A.ld_sc + b0 + b];
    }
    for (int e = threadIdx.x; e < nb * 16; e += 256) {
      const int b = e / 16, c = e % 16;
      sw[b][c] = w_sc[(WROWS ? (int64_t)min(n0 + c, A.N - 1) : n0 / 128) * A.ld_sc + b0 + b];
    }
#pragma unroll 1
    for (int at = wave; at < nb; at += 4 * RING) {
#pragma unroll
      for (int r = 0; r < RING; ++r) {
        if (at + 4 * r >= nb) continue;
        multiply(R[r], b0 + at + 4 * r, at + 4 * r);
        if (b0 + at + 4 * (r + RING) < nkb) load(R[r], b0 + at + 4 * (r + RING));
      }
    }
    lds_barrier();
    const int m = threadIdx.x >> 4, c = threadIdx.x & 15;
#pragma unroll 4
    for (int b = 0; b < nb; ++b)
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[i] = __builtin_fmaf(prod[b][i][m][c], sa[b][i * 16 + m] * sw[b][c], acc[i]);
    if (b0 + CH < nkb) lds_barrier();
  }
  const int m = threadIdx.x >> 4, c = threadIdx.x & 15;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    if (i * 16 + m >= rows || n0 + c >= A.N) continue;
    const int64_t at = (m0 + i * 16 + m) * A.N + n0 + c;
    if (A.bf16_out) static_cast<uint16_t*>(A.y)[at] = (uint16_t)bf16_pair(acc[i], 0.0f);
    else static_cast<float*>(A.y)[at] = acc[i];
  }
}

// ---------------------------------------------------------------------------
// Many rows: BM x BN tiles staged through LDS.  A stage holds one block of K
// of the tile's rows of both operands, brought by LDS DMA; WM x WN wavefronts
// of TM x TN 16 x 16 products each.  LDS rows are 128 bytes in 16-byte chunks,
// the chunk index XORed with the row's low bits, so that 8 rows' reads of one
// chunk fall on different banks.
template <int WM, int WN, int TM, int TN, int NST>
struct B128Shape {
  static constexpr int NW = WM * WN, BM = WM * TM * 16, BN = WN * TN * 16;
  static constexpr uint32_t OFF_W = BM * 128, STAGE = OFF_W + BN * 128, LDS = STAGE * NST;
  static constexpr int NX = BM / 8 / NW, NWT = BN / 8 / NW, NV = NX + NWT;    // DMA instructions per wavefront and stage
  static_assert(NX * NW * 8 == BM && NWT * NW * 8 == BN && LDS <= 160 * 1024 && NV * (NST - 1) < 63, "shape");
};

template <bool WROWS, B128Mode MODE, int WM, int WN, int TM, int TN, int NST>
__global__ __launch_bounds__(64 * WM * WN, 2) void b128_tile_kernel(B128Args A) {
  using S = B128Shape<WM, WN, TM, TN, NST>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4, wm = wave / WN, wn = wave % WN;
  const int nct = (int)(((int64_t)A.N + S::BN - 1) / S::BN);
  int64_t m0, y0 = 0;                             // first row of the operand; first result of the matrix
  int n0, rows, nkb = (A.K - 1) / 128 + 1, K = A.K;
  const uint8_t *x = A.a, *w = A.w;
  const float *x_sc = A.a_sc, *w_sc = A.w_sc;
  if (MODE == B128Mode::grouped) {
    // an XCD takes a row tile with all of its column tiles: its rows stay in that L2
    const uint32_t seq = blockIdx.x / XCDS, rt = seq / nct * XCDS + blockIdx.x % XCDS;
    const GroupTile t = find_tile(A.offsets, A.E, A.M, S::BM, rt);
    if (t.e < 0) return;
    m0 = t.row0 + (int64_t)t.tile * S::BM;
    rows = min(S::BM, t.rows - t.tile * S::BM);
    n0 = (int)(seq % nct) * S::BN;
    w += (int64_t)t.e * A.N * A.K;
    w_sc += (int64_t)t.e * ((A.N - 1) / 128 + 1) * nkb;
  } else {
    // XCD-aware order: each XCD takes a run of consecutive tiles, which go down 8 row tiles before the next column tile
    const int nrt = (int)(((int64_t)A.M + S::BM - 1) / S::BM);
    const uint32_t per_e = (uint32_t)nrt * nct, tiles = per_e * (MODE == B128Mode::wgrad ? A.E : 1), per = (tiles + XCDS - 1) / XCDS;
    uint32_t t = blockIdx.x % XCDS * per + blockIdx.x / XCDS;
    if (blockIdx.x / XCDS >= per || t >= tiles) return;
    if (MODE == B128Mode::wgrad) {
      const int e = (int)(t / per_e);
      t -= e * per_e;
      const GroupSpan s = find_span(A.offsets, A.E, A.ld, 128, e);
      const uint32_t all = (uint32_t)A.ld_sc, first = min(s.first, all);
      nkb = (int)min(s.n, all - first);
      K = nkb * 128;
      x += (int64_t)first * 128;
      w += (int64_t)first * 128;
      x_sc += first;
      w_sc += first;
      y0 = (int64_t)e * A.M * A.N;
    }
    const uint32_t grp = t / (8u * nct), in = t - grp * 8u * nct, rows_in = min(8u, nrt - grp * 8u);
    m0 = (int64_t)(grp * 8 + in % rows_in) * S::BM;
    n0 = (int)(in / rows_in) * S::BN;
    rows = (int)min((int64_t)S::BM, A.M - m0);
  }
  const int cols = min(S::BN, A.N - n0);
  x += m0 * A.ld;
  w += (int64_t)n0 * A.ld;
  x_sc += m0 * A.ld_sc;

  // this lane's DMA sources: rows past the last repeat it
  const uint8_t* xrow[S::NX];
  const uint8_t* wrow[S::NWT];
#pragma unroll
  for (int i = 0; i < S::NX; ++i) xrow[i] = x + min((i * S::NW + wave) * 8 + lane / 8, rows - 1) * A.ld;
#pragma unroll
  for (int i = 0; i < S::NWT; ++i) wrow[i] = w + min((i * S::NW + wave) * 8 + lane / 8, cols - 1) * A.ld;
  const int chunk = ((lane & 7) ^ (lane / 8)) * 16;                   // (row % 8 is lane / 8 in every instruction)
  auto issue = [&](int s) {
    uint8_t* const to = lds + (s % NST) * S::STAGE;
    const int k = min(s * 128 + chunk, K - 16);                       // past K: the row's last 16 again, cut later
#pragma unroll
    for (int i = 0; i < S::NX; ++i) dma16_to_lds(xrow[i] + k, to + (i * S::NW + wave) * 1024);
#pragma unroll
    for (int i = 0; i < S::NWT; ++i) dma16_to_lds(wrow[i] + k, to + S::OFF_W + (i * S::NW + wave) * 1024);
  };
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(lds));
  // zeros in the chunks of x past K, by the lane that brought them
  auto cut = [&](int s) {
    if (s * 128 + chunk < K) return;
#pragma unroll
    for (int i = 0; i < S::NX; ++i)
      lds_write(lds0 + (s % NST) * S::STAGE + (i * S::NW + wave) * 1024 + lane * 16, u32x4{0, 0, 0, 0});
  };
  const float* xs[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) xs[i] = x_sc + min((wm * TM + i) * 16 + col, rows - 1) * A.ld_sc;
  const float* ws[WROWS ? TN * 4 : 1];
  if (WROWS) {
#pragma unroll
    for (int j = 0; j < TN * 4; ++j) ws[WROWS ? j : 0] = w_sc + (int64_t)min(n0 + (wn * TN + j / 4) * 16 + 4 * g + j % 4, A.N - 1) * A.ld_sc;
  } else {
    static_assert(WROWS || 128 % (TN * 16) == 0, "one tile of weights per wavefront");
    ws[0] = w_sc + (int64_t)min((n0 + wn * TN * 16) / 128, (A.N - 1) / 128) * A.ld_sc;
  }
  float fx[TM], fw[WROWS ? TN * 4 : 1];
  auto fetch_scales = [&](int s) {
#pragma unroll
    for (int i = 0; i < TM; ++i) fx[i] = xs[i][s];
#pragma unroll
    for (int j = 0; j < (WROWS ? TN * 4 : 1); ++j) fw[j] = ws[j][s];
  };

  v4f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  const uint32_t xa = lds0 + (wm * TM * 16 + col) * 128, wa = lds0 + S::OFF_W + (wn * TN * 16 + col) * 128;
  const uint32_t c0 = (uint32_t)(g ^ (col & 7)) * 16, c1 = c0 ^ 64;

  if (nkb > 0) {
    fetch_scales(0);
#pragma unroll
    for (int s = 0; s < NST - 1; ++s)
      if (s < nkb) issue(s);
  }
  for (int s = 0; s < nkb; ++s) {
    if (NST > 2 && s + NST - 1 <= nkb) wait_vm<S::NV * (NST > 2 ? NST - 2 : 0)>();
    else wait_vm<0>();
    if (s == nkb - 1 && K % 128 != 0) cut(s);
    lds_barrier();
    float sx[TM], sw[WROWS ? TN * 4 : 1];
#pragma unroll
    for (int i = 0; i < TM; ++i) sx[i] = fx[i];
#pragma unroll
    for (int j = 0; j < (WROWS ? TN * 4 : 1); ++j) sw[j] = fw[j];
    if (s + 1 < nkb) fetch_scales(s + 1);
    if (s + NST - 1 < nkb) issue(s + NST - 1);
    const uint32_t buf = (s % NST) * S::STAGE;
    v8i xf[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i)
      xf[i] = operand8(lds_read<u32x4>(xa + buf + i * 2048 + c0), lds_read<u32x4>(xa + buf + i * 2048 + c1));
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const v8i wf = operand8(lds_read<u32x4>(wa + buf + j * 2048 + c0), lds_read<u32x4>(wa + buf + j * 2048 + c1));
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const v4f p = block_product(wf, xf[i]);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[i][j][r] = __builtin_fmaf(p[r], sx[i] * sw[WROWS ? j * 4 + r : 0], acc[i][j][r]);
      }
    }
  }

#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int m = (wm * TM + i) * 16 + col;
    if (m >= rows) continue;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int c = (wn * TN + j) * 16 + 4 * g;
      const int64_t at = y0 + (m0 + m) * A.N + n0 + c;
      const v4f& v = acc[i][j];
      if (c + 4 <= cols) {
        if (A.bf16_out) *reinterpret_cast<u32x2_a1*>(static_cast<uint16_t*>(A.y) + at) = u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
        else *reinterpret_cast<u32x4_a1*>(static_cast<float*>(A.y) + at) = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (c + r >= cols) continue;
          if (A.bf16_out) static_cast<uint16_t*>(A.y)[at + r] = (uint16_t)bf16_pair(v[r], 0.0f);
          else static_cast<float*>(A.y)[at + r] = v[r];
        }
      }
    }
  }
}

// Row tiles of `unit` that M rows in E groups can make.
static int64_t row_tiles(const B128Args& a, B128Mode mode, int unit) {
  if (mode != B128Mode::grouped) return ((int64_t)a.M + unit - 1) / unit;
  const int64_t e = a.E < a.M ? a.E : a.M;        // groups with rows
  return ((int64_t)a.M + (unit - 1) * e) / unit;
}

template <int MT, bool WROWS, B128Mode MODE> static void launch_rows(const B128Args& a, hipStream_t stream) {
  const int64_t n = row_tiles(a, MODE, 16 * MT) * (((int64_t)a.N + 15) / 16);
  hipLaunchKernelGGL((b128_rows_kernel<MT, WROWS, MODE>), dim3((unsigned)n), dim3(256), 0, stream, a);
}
// Workgroups of bm x bn tiles, in whole turns of the XCDs.
static int64_t tile_groups(const B128Args& a, B128Mode mode, int bm, int bn) {
  const int64_t nct = ((int64_t)a.N + bn - 1) / bn, n = row_tiles(a, mode, bm);
  if (mode == B128Mode::grouped) return (n + XCDS - 1) / XCDS * XCDS * nct;
  return (n * nct * (mode == B128Mode::wgrad ? a.E : 1) + XCDS - 1) / XCDS * XCDS;
}
template <bool WROWS, B128Mode MODE, int WM, int WN, int TM, int TN, int NST>
static void launch_tile(const B128Args& a, hipStream_t stream) {
  using S = B128Shape<WM, WN, TM, TN, NST>;
  hipLaunchKernelGGL((b128_tile_kernel<WROWS, MODE, WM, WN, TM, TN, NST>), dim3((unsigned)tile_groups(a, MODE, S::BM, S::BN)),
                     dim3(64 * S::NW), 0, stream, a);
}

enum class B128Kernel { rows16, rows32, t64x64, t128x128 };
static B128Kernel pick(const B128Args& a, B128Mode mode) {
  if (mode != B128Mode::wgrad) {
    const int64_t per = mode == B128Mode::grouped ? ((int64_t)a.M + a.E - 1) / a.E : a.M;   // rows of a matrix, about
    if (per <= 16) return B128Kernel::rows16;
    if (per <= 32) return B128Kernel::rows32;
  }
  if (mode == B128Mode::dense && tile_groups(a, mode, 128, 128) <= 256) return B128Kernel::t64x64;
  return B128Kernel::t128x128;
}

template <bool WROWS, B128Mode MODE> static const char* launch_of(const B128Args& a, hipStream_t stream) {
  switch (pick(a, MODE)) {
    case B128Kernel::rows16:
      if constexpr (MODE != B128Mode::wgrad) launch_rows<1, WROWS, MODE>(a, stream);
      return "b128:rows16";
    case B128Kernel::rows32:
      if constexpr (MODE != B128Mode::wgrad) launch_rows<2, WROWS, MODE>(a, stream);
      return "b128:rows32";
    case B128Kernel::t64x64:
      if constexpr (MODE == B128Mode::dense) launch_tile<WROWS, MODE, 2, 2, 2, 2, 4>(a, stream);
      return "b128:tile64x64";
    default: break;
  }
  launch_tile<WROWS, MODE, 2, 2, 4, 4, 2>(a, stream);
  return "b128:tile128x128";
}

// A launch holds fewer than 2^32 threads.
bool b128_fits(const B128Args& a, B128Mode mode) {
  switch (pick(a, mode)) {
    case B128Kernel::rows16: return row_tiles(a, mode, 16) * (((int64_t)a.N + 15) / 16) < int64_t(1) << 24;
    case B128Kernel::rows32: return row_tiles(a, mode, 32) * (((int64_t)a.N + 15) / 16) < int64_t(1) << 24;
    case B128Kernel::t64x64: return tile_groups(a, mode, 64, 64) < int64_t(1) << 24;
    default: return tile_groups(a, mode, 128, 128) < int64_t(1) << 24;
  }
}

hipError_t launch_b128(const B128Args& a, B128Mode mode, bool w_rows, hipStream_t stream, const char** variant) {
  if (mode == B128Mode::grouped) *variant = launch_of<false, B128Mode::grouped>(a, stream);
  else if (mode == B128Mode::wgrad) *variant = launch_of<true, B128Mode::wgrad>(a, stream);
  else if (w_rows) *variant = launch_of<true, B128Mode::dense>(a, stream);
  else *variant = launch_of<false, B128Mode::dense>(a, stream);
  return hipGetLastError();
}

}  // namespace mx
