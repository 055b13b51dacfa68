// Row groups of the grouped products (gfx950): which rows and which tile a
// workgroup has, from device offsets.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ufp4 {

__device__ __forceinline__ int64_t clamped(int64_t v, int64_t n) {
  return v < 0 ? 0 : (v > n ? n : v);
}

// A wave-uniform number in scalar registers.
__device__ __forceinline__ int64_t wave_uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// The group and the tile in it of tile t = pick(number of tiles), where group e has ceil(rows of e / bm)
// * per_row tiles.  Offsets are clamped to [0, M], a decreasing pair is an empty
// group.  Every wave finds it by itself: a lane sums a run of groups, a scan over
// the lanes finds the run, and the run is walked.
struct GroupTile {
  int e;                                         // -1: past the last tile
  int64_t row0, rows, local, tiles_m;
};
template <typename P>
__device__ __forceinline__ GroupTile find_tile(const int64_t *goff, int n_groups, int64_t M,
                                               int bm, int64_t per_row, P pick) {
  GroupTile g{0, 0, M, 0, (M + bm - 1) / bm};
  if (goff == nullptr) {
    g.local = pick(g.tiles_m * per_row);
    if (g.local >= g.tiles_m * per_row) g.e = -1;
    return g;
  }
  const int lane = threadIdx.x & 63;
  const int per = (n_groups + 63) / 64;
  auto tiles_of = [&](int e) -> int64_t {
    if (e >= n_groups) return 0;
    const int64_t n = clamped(goff[e + 1], M) - clamped(goff[e], M);
    return n > 0 ? (n + bm - 1) / bm : 0;
  };
  int64_t mine = 0;
  for (int i = 0; i < per; ++i) mine += tiles_of(lane * per + i);
  mine *= per_row;
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t v = __shfl_up(incl, o, 64);
    if (lane >= o) incl += v;
  }
  const int64_t t = pick((int64_t)__shfl(incl, 63, 64));
  const uint64_t over = __ballot(incl > t);
  if (over == 0) {
    g.e = -1;
    return g;
  }
  const int src = __builtin_ctzll(over);
  int64_t base = __shfl(incl - mine, src, 64);
  for (int e = src * per;; ++e) {
    const int64_t n = tiles_of(e);
    if (t < base + n * per_row) {
      g.e = e;
      g.row0 = clamped(goff[e], M);
      g.rows = clamped(goff[e + 1], M) - g.row0;
      g.local = t - base;
      g.tiles_m = n;
      return g;
    }
    base += n * per_row;
  }
}
// The same in scalar registers (every lane has found it, which the compiler cannot see).
template <typename P>
__device__ __forceinline__ GroupTile group_tile(const int64_t *goff, int n_groups, int64_t M,
                                                int bm, int64_t per_row, P pick) {
  const GroupTile g = find_tile(goff, n_groups, M, bm, per_row, pick);
  return {__builtin_amdgcn_readfirstlane(g.e), wave_uniform(g.row0), wave_uniform(g.rows),
          wave_uniform(g.local), wave_uniform(g.tiles_m)};
}

}  // namespace ufp4
