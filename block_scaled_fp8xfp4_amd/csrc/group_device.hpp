// Which expert a tile of rows belongs to, from the experts' row offsets on the
// device (moe_route's expert_offsets): found by every wavefront for itself,
// with one load of the offsets and one sum over its lanes, so that the host
// needs to know only a bound on the number of tiles.
#pragma once
#include "lds_device.hpp"

namespace mx {

// Sum over the lanes up to and with this one, by DPP (rows of 16, then rows 1 and 3, then the upper half).
__device__ __forceinline__ uint32_t lanes_upto(uint32_t v) {
  auto add = [&](auto ctrl, auto rows) {
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
  };
  add(Int<0x111>{}, Int<0xF>{});                  // row_shr:1
  add(Int<0x112>{}, Int<0xF>{});                  // row_shr:2
  add(Int<0x114>{}, Int<0xF>{});                  // row_shr:4
  add(Int<0x118>{}, Int<0xF>{});                  // row_shr:8
  add(Int<0x142>{}, Int<0xA>{});                  // row_bcast:15
  add(Int<0x143>{}, Int<0xC>{});                  // row_bcast:31
  return v;
}

struct GroupTile { int e, tile, row0, rows; };    // the expert, which of its tiles, its rows; e < 0: no such tile

// PER experts a lane (64 PER >= E).
template <int PER>
__device__ __forceinline__ GroupTile find_tile_of(const int32_t* offsets, int E, int64_t R, int unit, uint32_t t) {
  const int lane = fresh(threadIdx.x) & 63;
  int o[PER + 1];
  // what the offsets say is kept inside the R rows that there are
#pragma unroll
  for (int i = 0; i <= PER; ++i) o[i] = (int)max((int64_t)0, min((int64_t)offsets[min(lane * PER + i, E)], R));
  uint32_t n[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    n[i] = o[i + 1] > o[i] ? ((uint32_t)(o[i + 1] - o[i]) + (uint32_t)unit - 1) / (uint32_t)unit : 0u;
    sum += n[i];
  }
  const uint32_t upto = lanes_upto(sum);           // tiles up to and with this lane's
  const uint64_t past = __ballot(upto > t);
  if (past == 0) return GroupTile{-1, 0, 0, 0};
  uint32_t first = upto - sum;
  GroupTile g{-1, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (g.e < 0 && t < first + n[i]) g = GroupTile{lane * PER + i, (int)(t - first), o[i], o[i + 1] - o[i]};
    first += n[i];
  }
  const int src = __builtin_ctzll(past);
  g.e = __builtin_amdgcn_readlane(g.e, src);
  g.tile = __builtin_amdgcn_readlane(g.tile, src);
  g.row0 = __builtin_amdgcn_readlane(g.row0, src);
  g.rows = __builtin_amdgcn_readlane(g.rows, src);
  return g;
}
// The expert of tile t when each expert's rows are cut into tiles of `unit`.
// All 64 lanes of the wavefront take part.
__device__ __forceinline__ GroupTile find_tile(const int32_t* offsets, int E, int64_t R, int unit, uint32_t t) {
  return E <= 256 ? find_tile_of<4>(offsets, E, R, unit, t) : find_tile_of<16>(offsets, E, R, unit, t);
}

// Tiles [first, first + n) of expert e when each expert's rows are cut into tiles of `unit`.
struct GroupSpan { uint32_t first, n; };
template <int PER>
__device__ __forceinline__ GroupSpan find_span_of(const int32_t* offsets, int E, int64_t R, int unit, int e) {
  const int lane = fresh(threadIdx.x) & 63;
  uint32_t before = 0, mine = 0;
  int prev = (int)max((int64_t)0, min((int64_t)offsets[min(lane * PER, E)], R));
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int o = (int)max((int64_t)0, min((int64_t)offsets[min(lane * PER + i + 1, E)], R));
    const uint32_t n = o > prev ? ((uint32_t)(o - prev) + (uint32_t)unit - 1) / (uint32_t)unit : 0u;
    before += lane * PER + i < e ? n : 0u;
    mine += lane * PER + i == e ? n : 0u;
    prev = o;
  }
  return GroupSpan{(uint32_t)__builtin_amdgcn_readlane((int)lanes_upto(before), 63),
                   (uint32_t)__builtin_amdgcn_readlane((int)lanes_upto(mine), 63)};
}
__device__ __forceinline__ GroupSpan find_span(const int32_t* offsets, int E, int64_t R, int unit, int e) {
  return E <= 256 ? find_span_of<4>(offsets, E, R, unit, e) : find_span_of<16>(offsets, E, R, unit, e);
}

}  // namespace mx
