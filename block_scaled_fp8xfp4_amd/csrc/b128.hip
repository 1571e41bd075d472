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
//
// Precision: that step cuts E4M3 products below the largest of their eight
// (3.3e-5 of the result's norm on normal data; fp32 products of the decoded
// values 1e-7).  In bf16 it decides the rounding of 1.4 % of the results: with it
// and without they are 2.6e-4 of the norm apart, and 1.6559e-3 and 1.6558e-3 from
// the exact ones (8192 x 4096 x 4096).
#include "b128_launch.hpp"
#include "group_device.hpp"
#include "lds_device.hpp"
#include "mx_cast.hpp"

namespace mx {

typedef float v16f __attribute__((ext_vector_type(16)));

// W (A side: 16 rows n) x X (B side: 16 rows m), K = 128, from zero: lane l holds row m = l % 16 and columns
// n = 4 (l / 16) + [0, 4).
__device__ __forceinline__ v4f block_product(const v8i& w, const v8i& x) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ v8i operand8(const u32x4& lo, const u32x4& hi) {
  return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// ---------------------------------------------------------------------------
// Few rows: a workgroup per 16 columns and 16 MT rows.  Its four wavefronts
// take every fourth block of K, both operands straight to registers, and leave
// each block's products in LDS; then a thread per result adds them up in
// order.  What counts is bytes on their way: four workgroups per CU with RING
// blocks per wavefront.
template <int MT, bool WROWS, B128Mode MODE>
__global__ __launch_bounds__(256, 4) void b128_rows_kernel(B128Args A) {
  constexpr int CH = 32 / MT;                     // blocks of K whose products LDS holds at a time
  constexpr int RING = MT == 1 ? 4 : 2;
  constexpr int NS = CH * 16 * MT / 256, NC = CH * 16 / 256;  // rows' and columns' scales per thread and chunk
  static_assert(CH % (4 * RING) == 0 && NS * 256 == CH * 16 * MT && NC > 0, "chunks of whole rings, whole scales");
  __shared__ __attribute__((aligned(1024))) float prod[CH][MT][16][16];
  __shared__ float sa[CH][MT * 16], sw[WROWS ? CH : 1][16];           // rows' scales, times the tile's; WROWS: the columns'
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

  // scales of the chunk from block b0 on: thread's entries e = block, row (and column)
  float ra[NS], rw[NS], rc[WROWS ? NC : 1];
  auto fetch = [&](int b0) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int e = i * 256 + threadIdx.x, b = min(b0 + e / (16 * MT), nkb - 1), m = e % (16 * MT);
      ra[i] = A.a_sc[(m0 + min(m, rows - 1)) * A.ld_sc + b];
      rw[i] = WROWS ? 1.0f : w_sc[(int64_t)(n0 / 128) * A.ld_sc + b];
    }
    if (WROWS) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int e = i * 256 + threadIdx.x;
        rc[WROWS ? i : 0] = w_sc[min(n0 + e % 16, A.N - 1) * A.ld_sc + min(b0 + e / 16, nkb - 1)];
      }
    }
  };
  auto put = [&] {
#pragma unroll
    for (int i = 0; i < NS; ++i) (&sa[0][0])[i * 256 + threadIdx.x] = ra[i] * rw[i];
    if (WROWS) {
#pragma unroll
      for (int i = 0; i < NC; ++i) (&sw[0][0])[i * 256 + threadIdx.x] = rc[WROWS ? i : 0];
    }
  };

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
  fetch(0);
  __builtin_amdgcn_sched_barrier(0);              // the scales first: loads arrive in order
  Piece R[RING];
#pragma unroll
  for (int r = 0; r < RING; ++r)
    if (wave + 4 * r < nkb) load(R[r], wave + 4 * r);

  const int m = threadIdx.x >> 4, c = threadIdx.x & 15;
  float acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = 0.0f;
  for (int b0 = 0; b0 < nkb; b0 += CH) {
    const int nb = min(CH, nkb - b0);
    put();
    if (b0 + CH < nkb) fetch(b0 + CH);
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
#pragma unroll 8
    for (int b = 0; b < nb; ++b)
#pragma unroll
      for (int i = 0; i < MT; ++i)
        acc[i] = __builtin_fmaf(prod[b][i][m][c], WROWS ? sa[b][i * 16 + m] * sw[WROWS ? b : 0][c] : sa[b][i * 16 + m], acc[i]);
    if (b0 + CH < nkb) lds_barrier();
  }
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
// of the tile's rows of both operands and their scales, brought by LDS DMA;
// WM x WN wavefronts of TM x TN 16 x 16 products each.  LDS rows are 128 bytes
// in 16-byte chunks, the chunk index XORed with the row's low bits, so that 8
// rows' reads of one chunk fall on different banks.
//
// A wavefront walks over its TN columns of products: while one column's TM
// products are in the matrix cores, the column before is multiplied with its
// scales and added, and the column after is read from LDS.  The stage's one
// barrier comes before its last column, whose products cover the reads of the
// next stage's first operands; behind it the stage's buffer is free for DMA.

template <bool WROWS, int WM, int WN, int TM, int TN, int NST>
struct B128Shape {
  static constexpr int NW = WM * WN, BM = WM * TM * 16, BN = WN * TN * 16;
  // rows of scales, x's in whole 64s (a DMA instruction); surplus ones repeat the last
  static constexpr int XS = (BM + 63) / 64 * 64, NS = (XS + (WROWS ? BN : WN) + 64 * NW - 1) / (64 * NW);
  static constexpr uint32_t OFF_W = BM * 128, OFF_S = OFF_W + BN * 128, STAGE = OFF_S + NS * NW * 256;
  static constexpr uint32_t LDS = STAGE * NST;
  static constexpr int NX = BM / 8 / NW, NWT = BN / 8 / NW, NV = NX + NWT + NS;    // DMA instructions per wavefront and stage
  // DMA instructions go out one by one, two products apart, since a wavefront stalls at one while the memory path is still
  // taking the last: FIRST of them in the column that follows the barrier, the others over SPREAD products of the next stage
  static constexpr int FIRST = (TM + 1) / 2 < NV ? (TM + 1) / 2 : NV, REST = NV - FIRST;
  static constexpr int SPREAD = REST * 2 < (TN - 1) * TM ? REST * 2 : (TN - 1) * TM;
  static_assert(NX * NW * 8 == BM && NWT * NW * 8 == BN && LDS <= 160 * 1024 && NV * (NST - 1) < 63, "shape");
  static_assert(TN % 2 == 0 && (WROWS || 128 % (TN * 16) == 0), "pairs of columns; one tile of weights per wavefront");
};

template <bool WROWS, B128Mode MODE, int WM, int WN, int TM, int TN, int NST>
__global__ __launch_bounds__(64 * WM * WN, 2) void b128_tile_kernel(B128Args A) {
  using S = B128Shape<WROWS, WM, WN, TM, TN, NST>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4, wm = wave / WN, wn = wave % WN;
  const int nct = (int)(((int64_t)A.N + S::BN - 1) / S::BN);

  // The tile that the workgroup is at.
  int64_t m0, y0 = 0;                             // first row of the operand; first result of the matrix
  int n0, rows, cols, nkb, K;
  const uint8_t *x, *w;
  const float *xs, *ws;
  // this lane's DMA sources, from the tile's first row on: rows past the last repeat it
  uint32_t xoff[S::NX], woff[S::NWT], soff[S::NS];
  const int chunk = ((lane & 7) ^ (lane / 8)) * 16;                   // (row % 8 is lane / 8 in every instruction)
  const uint32_t seq = blockIdx.x / XCDS;         // of this XCD's tiles
  xs = A.a_sc;
  ws = A.w_sc;
  x = A.a;
  w = A.w;
  K = A.K;
  nkb = (K - 1) / 128 + 1;
  if (MODE == B128Mode::grouped) {
    // an XCD takes a row tile with all of its column tiles: its rows stay in that L2
    const uint32_t rt = seq / nct * XCDS + blockIdx.x % XCDS;
    const GroupTile t = find_tile(A.offsets, A.E, A.M, S::BM, rt);
    if (t.e < 0) return;
    m0 = t.row0 + (int64_t)t.tile * S::BM;
    rows = min(S::BM, t.rows - t.tile * S::BM);
    n0 = (int)(seq % nct) * S::BN;
    w += (int64_t)t.e * A.N * A.K;
    ws += (int64_t)t.e * ((A.N - 1) / 128 + 1) * nkb;
  } else {
    // XCD-aware order: each XCD takes a run of consecutive tiles, which go down 8 row tiles before the next column tile
    const int nrt = (int)(((int64_t)A.M + S::BM - 1) / S::BM);
    const uint32_t per_e = (uint32_t)nrt * nct, tiles = per_e * (MODE == B128Mode::wgrad ? A.E : 1), per = (tiles + XCDS - 1) / XCDS;
    uint32_t t = blockIdx.x % XCDS * per + seq;
    if (seq >= per || t >= tiles) return;
    if (MODE == B128Mode::wgrad) {
      const int e = (int)(t / per_e);
      t -= e * per_e;
      const GroupSpan s = find_span(A.offsets, A.E, A.ld, 128, e);
      const uint32_t all = (uint32_t)A.ld_sc, first = min(s.first, all);
      nkb = (int)min(s.n, all - first);
      K = nkb * 128;
      x += (int64_t)first * 128;
      w += (int64_t)first * 128;
      xs += first;
      ws += first;
      y0 = (int64_t)e * A.M * A.N;
    }
    const uint32_t grp = t / (8u * nct), in = t - grp * 8u * nct, rows_in = min(8u, nrt - grp * 8u);
    m0 = (int64_t)(grp * 8 + in % rows_in) * S::BM;
    n0 = (int)(in / rows_in) * S::BN;
    rows = (int)min((int64_t)S::BM, A.M - m0);
  }
  rows = __builtin_amdgcn_readfirstlane(rows);
  n0 = __builtin_amdgcn_readfirstlane(n0);
  cols = min(S::BN, A.N - n0);
  x += m0 * A.ld;
  w += (int64_t)n0 * A.ld;
  xs += m0 * A.ld_sc;
  ws += (int64_t)(WROWS ? n0 : n0 / 128) * A.ld_sc;
#pragma unroll
  for (int i = 0; i < S::NX; ++i) xoff[i] = (uint32_t)min((i * S::NW + wave) * 8 + lane / 8, rows - 1) * (uint32_t)A.ld + (uint32_t)chunk;
#pragma unroll
  for (int i = 0; i < S::NWT; ++i) woff[i] = (uint32_t)min((i * S::NW + wave) * 8 + lane / 8, cols - 1) * (uint32_t)A.ld + (uint32_t)chunk;
#pragma unroll
  for (int i = 0; i < S::NS; ++i) {
    const int r = (i * S::NW + wave) * 64 + lane, c = min(r - S::XS, WROWS ? S::BN - 1 : WN - 1);
    const int wr = WROWS ? min(c, cols - 1) : (n0 % 128 + min(c * TN * 16, cols - 1)) / 128;
    soff[i] = (uint32_t)(r < S::XS ? min(r, rows - 1) : wr) * (uint32_t)A.ld_sc * 4;
  }
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(lds));
  // the d-th DMA instruction of stage s; past: what this lane's chunk reaches past K (the row's last 16 are read again, and
  // cut when they have landed)
  auto issue1 = [&](int s, uint32_t buf, int d, uint32_t past) {
    const int ix = min(max(d - S::NS, 0), S::NX - 1), iw = max(d - S::NS - S::NX, 0);
    if (d < S::NS)                                // 64 rows of scales are all x's or all w's
      dma4_to_lds(((d * S::NW + wave) * 64 < S::XS ? xs : ws) + s, soff[min(d, S::NS - 1)], lds0 + buf + S::OFF_S + (d * S::NW + wave) * 256);
    else if (d < S::NS + S::NX) dma16_to_lds(x + (int64_t)s * 128, xoff[ix] - past, lds0 + buf + (ix * S::NW + wave) * 1024);
    else dma16_to_lds(w + (int64_t)s * 128, woff[iw] - past, lds0 + buf + S::OFF_W + (iw * S::NW + wave) * 1024);
  };
  auto reach = [&] {                              // past K in the last stage
    const int lane = fresh(threadIdx.x) & 63;
    return max((nkb - 1) * 128 + ((lane & 7) ^ (lane / 8)) * 16 - (K - 16), 0);
  };
  auto issue = [&](int s, uint32_t buf, int d0, int d1) {
    const uint32_t past = s == nkb - 1 ? reach() : 0;
#pragma unroll
    for (int d = d0; d < d1; ++d) issue1(s, buf, d, past);
  };
  // zeros in the chunks of x past K, by the lane that brought them
  auto cut = [&](int s, uint32_t buf) {
    if (s != nkb - 1 || K % 128 == 0 || reach() == 0) return;
#pragma unroll
    for (int i = 0; i < S::NX; ++i) lds_write(lds0 + buf + (i * S::NW + wave) * 1024 + (fresh(threadIdx.x) & 63) * 16, u32x4{0, 0, 0, 0});
  };
  // Stage s has landed for this wavefront (later ones, as many as were asked for, may be on their way).
  auto landed = [&](int s, uint32_t buf) {
    if (NST > 2 && s + NST - 2 < nkb) wait_vm<S::NV * (NST > 2 ? NST - 2 : 0)>();
    else wait_vm<0>();
    cut(s, buf);
    lds_barrier();
  };
  auto before = [](uint32_t buf) { return buf == 0 ? (NST - 1) * S::STAGE : buf - S::STAGE; };
  auto after = [](uint32_t buf) { return buf + S::STAGE == NST * S::STAGE ? 0u : buf + S::STAGE; };

  const uint32_t xa = lds0 + (wm * TM * 16 + col) * 128, wa = lds0 + S::OFF_W + (wn * TN * 16 + col) * 128;
  const uint32_t c0 = (uint32_t)(g ^ (col & 7)) * 16, c1 = c0 ^ 64;

  v4f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  if (nkb > 0) {
#pragma unroll
    for (int s = 0; s + 1 < NST; ++s)
      if (s < nkb) issue(s, s * S::STAGE, 0, S::NV);
    if (NST - 1 < nkb) issue(NST - 1, (NST - 1) * S::STAGE, 0, S::FIRST);
    // the first stage: as landed(0), with part of one stage more on its way
    if (nkb >= NST) wait_vm<S::NV * (NST - 2) + S::FIRST>();
    else wait_vm<0>();
    cut(0, 0);
    lds_barrier();
    // nothing of this wavefront's is a result (256 experts' 1152 x 4096, 8192 x 8 rows: 535 us, 552 with products of columns past N)
    if (wm * TM * 16 >= rows || wn * TN * 16 >= cols) {
      uint32_t buf = 0;
      if (NST - 1 < nkb) issue(NST - 1, (NST - 1) * S::STAGE, S::FIRST, S::NV);
      for (int s = 0; s + 1 < nkb; ++s) {
        landed(s + 1, after(buf));
        if (s + NST < nkb) issue(s + NST, buf, 0, S::NV);
        buf = after(buf);
      }
    } else {
      v8i xf[TM], wf[2];                          // operands of a column of products: this one's and the next one's
      v4f P[2][TM];                               // products on their way, and those of the column before
      // OUTER: the matrix cores multiply the scales too, a column's 16 with the 64 of the rows, in fp32 as the vector unit
      // does, bit for bit; a lane holds one of each.  It halves the vector instructions beside the products where both operands
      // have scales by rows: 8192 x 4096 x 4096 again and again 170 us from 183 (with pauses 148), 4096 x 2048 x 8192 91 from 95,
      // 64 experts' gradients 1152 x 2048 of 4096 x 8 rows 175 from 178
      constexpr bool OUTER = WROWS && TM == 4;
      float f[TM], fn[TM], wn_ = 0.f;             // scales of the rows (times the tile's): the stage's, the next one's
      v4f sn{};                                   // WROWS: scales of the column's weight rows
      v16f prods{};                               // OUTER: scales of the column before, all TM x 4
      auto load_x = [&](int i, uint32_t buf) {
        xf[i] = operand8(lds_read<u32x4>(xa + c0 + buf + i * 2048), lds_read<u32x4>(xa + c1 + buf + i * 2048));
      };
      auto load_w = [&](int j, uint32_t buf) {
        wf[j & 1] = operand8(lds_read<u32x4>(wa + c0 + buf + j * 2048), lds_read<u32x4>(wa + c1 + buf + j * 2048));
      };
      auto load_scales = [&](uint32_t buf) {
#pragma unroll
        for (int i = 0; i < (OUTER ? 1 : TM); ++i)
          fn[i] = lds_read<float>(lds0 + buf + S::OFF_S + ((wm * TM + i) * 16 + (OUTER ? lane : col)) * 4);
        if (!WROWS) wn_ = lds_read<float>(lds0 + buf + S::OFF_S + (S::XS + wn) * 4);
      };
      // Holds the sums before the branches that follow (no instruction): the compiler would move them behind.
      auto pin = [&] {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) asm volatile("" : "+v"(acc[i][j]));
      };
      // Stage s.  MORE 0: there is none after it; 1: there is, and maybe stages to ask for; 2: there are NST + 1 whole ones.
      auto stage = [&](int s, uint32_t buf, auto more) {
        constexpr int MORE = decltype(more)::value;
        const uint32_t nbuf = after(buf);
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const bool end = j == TN - 1;
          const v4f sp = sn;                      // of the column before
          if (OUTER) sn[0] = lds_read<float>(lds0 + buf + S::OFF_S + (S::XS + (wn * TN + j) * 16 + col) * 4);
          else if (WROWS) sn = lds_read<v4f>(lds0 + buf + S::OFF_S + (S::XS + (wn * TN + j) * 16 + 4 * g) * 4);
          if (end && MORE == 1) {
            pin();
            landed(s + 1, nbuf);
            if (s + NST < nkb) issue(s + NST, buf, 0, S::NV);
          }
          if (end && MORE == 2) {
            wait_vm<S::NV * (NST - 2)>();
            lds_barrier();
          }
          if (!end) load_w(j + 1, buf);
          else if (MORE) {
            load_w(0, nbuf);
            load_scales(nbuf);
          }
#pragma unroll
          for (int i = 0; i < TM; ++i) {
            P[j & 1][i] = block_product(wf[j & 1], xf[i]);
            const int jp = j == 0 ? TN - 1 : j - 1;
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[i][jp][r] = __builtin_fmaf(P[jp & 1][i][r], OUTER ? prods[i * 4 + r] : WROWS ? f[i] * sp[r] : f[i], acc[i][jp][r]);
            if (end && MORE) load_x(i, nbuf);
            if (end && MORE == 2 && i % 2 == 0 && i / 2 < S::FIRST) issue1(s + NST, buf, i / 2, 0);
            if (!end && MORE == 2 && j * TM + i < S::SPREAD) {
#pragma unroll
              for (int d = (j * TM + i) * S::REST / S::SPREAD; d < (j * TM + i + 1) * S::REST / S::SPREAD; ++d)
                issue1(s + NST - 1, before(buf), S::FIRST + d, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
          if (j == 0) {
#pragma unroll
            for (int i = 0; i < (OUTER ? 1 : TM); ++i) f[i] = WROWS ? fn[i] : fn[i] * wn_;
          }
          if (OUTER) {
            prods = __builtin_amdgcn_mfma_f32_16x16x1f32(sn[0], f[0], v16f{}, 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      };
      // before the first column: products of zero
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        P[(TN - 1) & 1][i] = v4f{0.f, 0.f, 0.f, 0.f};
        f[i] = 0.f;
        load_x(i, 0);
      }
      load_w(0, 0);
      load_scales(0);
      uint32_t buf = 0;
      int s = 0;
      for (const int whole = K / 128; s + NST < whole; ++s) {
        stage(s, buf, Int<2>{});
        buf = after(buf);
      }
      if (s + NST - 1 < nkb) issue(s + NST - 1, before(buf), S::FIRST, S::NV);
      for (; s + 1 < nkb; ++s) {
        stage(s, buf, Int<1>{});
        buf = after(buf);
      }
      stage(s, buf, Int<0>{});
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[i][TN - 1][r] = __builtin_fmaf(P[(TN - 1) & 1][i][r], OUTER ? prods[i * 4 + r] : WROWS ? f[i] * sn[r] : f[i], acc[i][TN - 1][r]);
    }
  }

  // Results.  Each wavefront turns 16 rows of 128 bytes at a time in its own part of LDS, so that a store instruction writes
  // whole runs of a row: 16 bytes a lane, at whatever alignment the row has, the row's last piece by elements.
  lds_barrier();                                                      // every wavefront has read its operands
  const int nw = min(TN * 16, cols - wn * TN * 16);                   // this wavefront's columns
  const int64_t y_ = y0 + m0 * A.N + n0 + wn * TN * 16;
  constexpr uint32_t PITCH = 128 + 16;                                // + 16: rows start on different banks
  const int lane_ = fresh(threadIdx.x) & 63, col_ = lane_ & 15, g_ = lane_ >> 4;
  const uint32_t mine = lds0 + wave * 16 * PITCH;
  static_assert(S::NW * 16 * PITCH <= S::LDS, "results in LDS");
  auto store = [&](auto esize, auto far) {                            // bytes of a result; past the caches
    constexpr int ESZ = decltype(esize)::value, PER = 16 / ESZ;       // elements per lane
    constexpr int JS = TN * 16 * ESZ < 128 ? TN : 128 / ESZ / 16, LPR = JS * 16 * ESZ / 16;   // products and lanes per run
    constexpr int RPP = 64 / LPR, PASSES = 16 / RPP;                  // rows at a time
    const int r0 = lane_ / LPR, c = lane_ % LPR * PER;
    const uint32_t from = mine + r0 * PITCH + c * ESZ;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int mb = (wm * TM + i) * 16;
      if (mb >= rows) break;
#pragma unroll
      for (int j0 = 0; j0 < TN; j0 += JS) {
#pragma unroll
        for (int j = j0; j < j0 + JS; ++j) {
          const v4f& v = acc[i][j];
          const uint32_t at = mine + col_ * PITCH + ((j - j0) * 16 + 4 * g_) * ESZ;
          if (ESZ == 2) lds_write(at, u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])});
          else lds_write(at, v);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");            // the wavefront's own writes
        uint8_t* to = static_cast<uint8_t*>(A.y) + (y_ + (int64_t)(mb + r0) * A.N + j0 * 16 + c) * ESZ;
#pragma unroll
        for (int p = 0; p < PASSES; ++p, to += (int64_t)RPP * A.N * ESZ) {
          const u32x4 d = lds_read<u32x4>(from + p * RPP * PITCH);
          if (mb + r0 + p * RPP >= rows) continue;
          if (j0 * 16 + c + PER <= nw) {
            if constexpr (decltype(far)::value) __builtin_nontemporal_store(d, reinterpret_cast<u32x4_a1*>(to));
            else *reinterpret_cast<u32x4_a1*>(to) = d;
          } else
#pragma unroll
            for (int e = 0; e < PER; ++e) {
              if (j0 * 16 + c + e >= nw) continue;
              if (ESZ == 2) reinterpret_cast<uint16_t*>(to)[e] = (uint16_t)(d[e / (4 / ESZ)] >> (16 * (e % 2)));
              else reinterpret_cast<uint32_t*>(to)[e] = d[e / (4 / ESZ)];
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      }
    }
  };
  if (A.far) {
    if (A.bf16_out) store(Int<2>{}, Int<1>{});
    else store(Int<4>{}, Int<1>{});
  } else {
    if (A.bf16_out) store(Int<2>{}, Int<0>{});
    else store(Int<4>{}, Int<0>{});
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

// Which kernel, by how many workgroups each shape gives and what a round of them takes.  us, weights from memory:
//   rows of 4096 x 4096:    1 rows16 8.2, 64 x 64 11.4; 32 rows32 9.8, 64 x 64 12.0; 48 64 x 64 13.5, rows32 13.7
//           16384 x 4096:   1 16 x 64 16.1, rows16 18.8 (DMA keeps more bytes on their way than registers); 9216 x 4096: 16 16 x 64
//                           12.2, 64 x 64 13.6; 8192 x 4096: 1 rows16 9.9, 16 x 64 11.4; 129280 x 4096: 1 16 x 64 98.7, 128 x 256 104.5
//           1152 x 4096:    48 rows16 7.1, 64 x 64 10.2; 96 rows32 8.7, 64 x 64 10.3
//           4096 x 4096:    256 64 x 64 14.9, 64 x 128 20.5; 512 64 x 128 18.6, 64 x 64 23.3; 700 128 x 128 22.3, 64 x 256 28.2; 1024
//                           128 x 128 29.6, 64 x 128 32.2, 64 x 256 32.3, 128 x 256 36.9; 2048 128 x 256 41.2, 256 x 256 59.6; 4096 256 x 256 68.0, 128 x 256 79.5
//   256 experts' 1152 x 4096, rows each: 4 64 x 64 209, 64 x 128 225, rows16 248; 32 64 x 128 248, 64 x 64 254, 128 x 256 259;
//                           64 128 x 256 275, 64 x 128 295; 192 256 x 256 395, 128 x 256 439; 256 256 x 256 492, 128 x 256
//                           510
//                           8 rows of all 16 x 64 13.3, 64 x 64 15.7; 32 rows 30.3, 35.5; 64 56.5, 60.7; 384 179, 180; 1024 215, 214;
//                           2048 224, 219 (16 x 64 in 8 stages, one workgroup a CU: 12.6, 36.4, 61, 189, 232, 236)
//   8 experts' 4096 x 4096, rows each: 8 64 x 128 21.0, 64 x 64 21.1, 128 x 256 22.4; 64 128 x 256 30.1, 64 x 128 40.5; 128
//                           128 x 256 37.7, 256 x 256 47.5; 256 256 x 256 60, 128 x 256 71; 1024 192, 208
//   64 experts' 1152 x 2048, rows each: 128 128 x 256 44, 256 x 256 51; 256 256 x 256 73, 128 x 256 79; 512 128, 138
//   gradients, 1024 tokens each, by workgroups of 128 x 128: 8 experts' 512 x 1024 (256) 128 x 128 13.1, 256 x 256 22.7; 640 x 1024
//                           (320) 23.4, 23.4; 12 of 512 x 1024 (384) 24.7, 25.8; 16 (512) 26.2, 26.8; 32 (1024) 48.8, 30.1
//   256 experts, 64 x 64 and 64 x 128, 4 and 16 rows each: 1152 x 2048 104, 101 and 112, 108; x 2304 116, 114 and 126, 124; x 3328
//                           163, 162 and 178, 174; x 4096 212, 228 and 223, 237; x 5120 246, 247 and 275, 266; 512 x 2304 58.4, 53.9;
//                           64 experts of 3 rows x 2048 31.6, 32.7; x 2816 42.5, 44.0; x 4096 65.7, 73.3: the border of K lies where
//                           neither is ahead by more than 3 % (8 at 512 columns)
//                           12 rows each, K = 2048: 64 columns 10.9, 12.4; 128 16.6, 17.1; 256 29.6, 29.0
//   scales by rows on both sides, K = 4096, 128 x 256 and 256 x 256: 2048 x 4096 49.6, 63.9; 2560 76.2, 65.0; 5120 117.7, 124.5; 6144
//                           128.6, 128.0; 8192 183.6, 146.4
//   256 experts' 1152 x 4096 chosen as 1 / rank: 8192 x 8 rows 256 x 256 501, 128 x 256 500; 2048 x 8 128 x 256 291, 64 x 128 299,
//                           256 x 256 333; 512 x 8 64 x 64 227, 64 x 128 237
//   256 experts' 4096 x 576, 48 rows of all: 64 x 128 95, 64 x 64 126, rows16 187 (few blocks of K: what a workgroup begins
//                           and ends with counts)
enum class B128Kernel { rows16, rows32, t16x64, t64x64, t64x128, t128x128, t128x256, t256x256 };
struct B128Group { int rows, cols, threads; };                        // of a workgroup
static constexpr B128Group group_of(B128Kernel k) {
  switch (k) {
    case B128Kernel::rows16: return {16, 16, 256};
    case B128Kernel::rows32: return {32, 16, 256};
    case B128Kernel::t16x64: return {16, 64, 128};
    case B128Kernel::t64x64: return {64, 64, 256};
    case B128Kernel::t64x128: return {64, 128, 512};
    case B128Kernel::t128x128: return {128, 128, 512};
    case B128Kernel::t128x256: return {128, 256, 512};
    default: return {256, 256, 512};
  }
}
// A launch holds fewer than 2^32 threads.
static bool launch_holds(const B128Args& a, B128Mode mode, B128Kernel k) {
  const B128Group g = group_of(k);
  return tile_groups(a, mode, g.rows, g.cols) < (int64_t(1) << 32) / g.threads;
}
static int64_t row_groups(const B128Args& a, B128Mode mode, int rows) { return row_tiles(a, mode, rows) * (((int64_t)a.N + 15) / 16); }
// Workgroups with rows that experts of about as many rows each make: half a tile more than whole ones, at least one each.
static int64_t likely_groups(const B128Args& a, int bm, int bn) {
  const int64_t e = a.E < a.M ? a.E : a.M, n = ((int64_t)a.M + (e - 1) * (bm / 2) + bm - 1) / bm;
  return (n > e ? n : e) * (((int64_t)a.N + bn - 1) / bn);
}
static B128Kernel quickest(const B128Args& a, B128Mode mode) {
  if (mode == B128Mode::wgrad) return tile_groups(a, mode, 128, 128) <= 256 ? B128Kernel::t128x128 : B128Kernel::t256x256;
  if (row_groups(a, mode, 16) <= 256) return B128Kernel::rows16;
  if (mode == B128Mode::grouped) {
    if (row_groups(a, mode, 16) <= 512) return B128Kernel::rows16;
    if (a.M <= 2 * (int64_t)a.E) return B128Kernel::t16x64;           // two rows each, three workgroups a CU
    if (likely_groups(a, 64, 64) <= 256) return B128Kernel::t64x64;
    if (likely_groups(a, 64, 128) <= 256) return B128Kernel::t64x128;
    const int64_t per = ((int64_t)a.M + a.E - 1) / a.E;               // rows of an expert, about; most fit one tile
    if (per <= 44) return per <= 24 && (a.K > 2048 || a.N <= 64) ? B128Kernel::t64x64 : B128Kernel::t64x128;
    // rounds of the largest two, at 3 to 2 (tiles of 256 rows are less full); past the second they run into one another
    auto rounds = [](int64_t n) { return n <= 512 ? (n + 255) / 256 * 256 : n; };
    return rounds(likely_groups(a, 256, 256)) * 3 <= rounds(likely_groups(a, 128, 256)) * 2 ? B128Kernel::t256x256 : B128Kernel::t128x256;
  }
  if (a.M > 16 && row_groups(a, mode, 32) <= 256) return B128Kernel::rows32;
  if (a.M <= 16 && row_groups(a, mode, 16) <= 512) return B128Kernel::rows16;
  if (a.M <= 16) return B128Kernel::t16x64;                           // one row of tiles, three workgroups a CU
  // the smallest tiles that are one round; past them rounds of the largest two, at 5 to 3
  if (tile_groups(a, mode, 64, 64) <= 256) return B128Kernel::t64x64;
  if (tile_groups(a, mode, 64, 128) <= 256) return B128Kernel::t64x128;
  if (tile_groups(a, mode, 128, 128) <= 256) return B128Kernel::t128x128;
  return (tile_groups(a, mode, 256, 256) + 255) / 256 * 5 <= (tile_groups(a, mode, 128, 256) + 255) / 256 * 3 ? B128Kernel::t256x256
                                                                                                              : B128Kernel::t128x256;
}

// Where one launch does not hold the quickest kernel's workgroups (1024 experts' few rows by 2^20 columns), larger tiles;
// weight gradients have no others.
static B128Kernel pick(const B128Args& a, B128Mode mode) {
  const B128Kernel k = quickest(a, mode);
  if (launch_holds(a, mode, k)) return k;
  return mode != B128Mode::wgrad && launch_holds(a, mode, B128Kernel::t128x256) ? B128Kernel::t128x256 : B128Kernel::t256x256;
}
bool b128_fits(const B128Args& a, B128Mode mode) { return launch_holds(a, mode, pick(a, mode)); }

template <bool WROWS, B128Mode MODE, B128Kernel KERNEL, int WM, int WN, int TM, int TN, int NST>
static void launch_tile(const B128Args& a, hipStream_t stream) {
  using S = B128Shape<WROWS, WM, WN, TM, TN, NST>;
  constexpr B128Group G = group_of(KERNEL);
  static_assert(G.rows == S::BM && G.cols == S::BN && G.threads == 64 * S::NW, "what the limits are counted by");
  const int64_t n = tile_groups(a, MODE, S::BM, S::BN);
  hipLaunchKernelGGL((b128_tile_kernel<WROWS, MODE, WM, WN, TM, TN, NST>), dim3((unsigned)n), dim3(64 * S::NW), 0, stream, a);
}
template <bool WROWS, B128Mode MODE> static const char* launch_of(const B128Args& a, hipStream_t stream) {
  using K = B128Kernel;
  const K k = pick(a, MODE);
  if constexpr (MODE != B128Mode::wgrad) {
    switch (k) {
      case K::rows16: launch_rows<1, WROWS, MODE>(a, stream); return "b128:rows16";
      case K::t16x64: launch_tile<WROWS, MODE, K::t16x64, 1, 2, 1, 2, 5>(a, stream); return "b128:tile16x64";
      case K::t64x64: launch_tile<WROWS, MODE, K::t64x64, 2, 2, 2, 2, 4>(a, stream); return "b128:tile64x64";
      case K::t64x128: launch_tile<WROWS, MODE, K::t64x128, 2, 4, 2, 2, MODE == B128Mode::dense ? 4 : 3>(a, stream); return "b128:tile64x128";
      case K::t128x256: launch_tile<WROWS, MODE, K::t128x256, 2, 4, 4, 4, 3>(a, stream); return "b128:tile128x256";
      default: break;
    }
  }
  if constexpr (MODE == B128Mode::dense)
    if (k == K::rows32) { launch_rows<2, WROWS, MODE>(a, stream); return "b128:rows32"; }
  if constexpr (MODE != B128Mode::grouped)
    if (k == K::t128x128) { launch_tile<WROWS, MODE, K::t128x128, 2, 4, 4, 2, 4>(a, stream); return "b128:tile128x128"; }
  launch_tile<WROWS, MODE, K::t256x256, 4, 2, 4, 8, 2>(a, stream);
  return "b128:tile256x256";
}

// Results of more than 64 MB go past the caches: nothing finds them there, and what they would push out is read again
// (64 experts' 1152 x 2048 gradients of 512 tokens each 172 us from 199, 256 experts' rows of 8192 x 8 by 1152 x 4096 504
// from 515).
static bool far_results(const B128Args& a, B128Mode mode) {
  return (int64_t)a.M * a.N * (mode == B128Mode::wgrad ? a.E : 1) * (a.bf16_out ? 2 : 4) > int64_t(64) << 20;
}

hipError_t launch_b128(B128Args a, B128Mode mode, bool w_rows, hipStream_t stream, const char** variant) {
  a.far = far_results(a, mode);
  if (mode == B128Mode::grouped) *variant = launch_of<false, B128Mode::grouped>(a, stream);
  else if (mode == B128Mode::wgrad) *variant = launch_of<true, B128Mode::wgrad>(a, stream);
  else if (w_rows) *variant = launch_of<true, B128Mode::dense>(a, stream);
  else *variant = launch_of<false, B128Mode::dense>(a, stream);
  return hipGetLastError();
}

}  // namespace mx
