// Device helpers shared by the kernels over expert-sorted rows: an expert's rows, and the tile
// or expert that a workgroup works on, found by every wave on its own from the offsets (no LDS,
// no barrier, one round of loads).
#pragma once

#include "moe_internal.h"

namespace moe {

// Rows [a, b) of expert e, with the offsets clamped into [0, rows] and made non-decreasing so
// that corrupt offsets can never address memory out of bounds.
__device__ __forceinline__ void group_rows(const int32_t* offsets, int e, int rows, int& a, int& b) {
  a = offsets[e];
  b = offsets[e + 1];
  a = a < 0 ? 0 : (a > rows ? rows : a);
  b = b < a ? a : (b > rows ? rows : b);
}

// Rows in use: offsets[E] when the caller gave the offsets (rows past it belong to no expert
// and are neither read nor written), else all of them.
__device__ __forceinline__ int rows_in_use(const int32_t* offsets, int E, int rows) {
  if (!offsets) return rows;
  const int n = offsets[E];
  return n < 0 ? 0 : (n > rows ? rows : n);
}

// Workgroup b's item of `items`, or -1. The hardware deals workgroups to the 8 XCDs in turn
// (workgroup b runs on XCD b % 8) and each XCD has an L2 of its own: every 256 workgroups take 256
// consecutive items, and each XCD a run of 32 of them, which share operands; a last, smaller round
// is cut into 8 runs as well, so that it keeps every XCD busy.
constexpr int kRound = 256;
__device__ __forceinline__ int xcd_item(unsigned b, unsigned items) {
  const unsigned base = b & ~(kRound - 1u);
  if (base >= items) return -1;
  const unsigned n = min((unsigned)kRound, items - base), run = (n + 7) / 8;
  const unsigned i = (b - base) >> 3, at = (b & 7) * run + i;
  return i < run && at < n ? (int)(base + at) : -1;
}
// Workgroups that meet all of `items` under that map.
inline long long xcd_grid(long long items) { return (items + kRound - 1) / kRound * kRound; }

// Tile pair of the i-th of mtiles * NT tiles: groups of kGroupM row tiles walk the column tiles
// together, so that the tiles in flight on one XCD share both operands.
constexpr int kGroupM = 4;
__device__ __forceinline__ void tile_pair(int i, int mtiles, int NT, int& mt, int& nt) {
  const int g = i / (kGroupM * NT);
  const int gm = min(kGroupM, mtiles - g * kGroupM);
  const int j = i - g * kGroupM * NT;
  nt = j / gm;
  mt = g * kGroupM + j % gm;
}

// Row tiles of TM rows, expert by expert; each of an expert's row tiles meets NT column tiles.
// Finds this workgroup's item: its expert e, the expert's rows [a, b) and the tile pair (mt, nt)
// within the expert; false if there is none.
__device__ __forceinline__ bool find_row_tile(const int32_t* offsets, int E, int rows, int TM,
                                              int NT, int& e, int& a, int& b, int& mt, int& nt) {
  const int lane = threadIdx.x & 63;
  const int per = (E + 63) / 64;  // consecutive experts per lane
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int x = lane * per + i;
    if (x < E) {
      int p, q;
      group_rows(offsets, x, rows, p, q);
      mine += (q - p + TM - 1) / TM;
    }
  }
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d);
    if (lane >= d) incl += v;
  }
  const int item = xcd_item(blockIdx.x, (unsigned)__builtin_amdgcn_readlane(incl, 63) * (unsigned)NT);
  if (item < 0) return false;
  const int q = item / NT;
  const unsigned long long past = __ballot(incl > q);  // never empty: q < all tiles
  const int owner = __ffsll(past) - 1;
  int pre = __builtin_amdgcn_readlane(incl - mine, owner);
  // the owner's experts, read by every lane (uniform addresses)
  e = owner * per;
  int mtiles = 0;
  for (;; ++e) {
    group_rows(offsets, e, rows, a, b);
    mtiles = __builtin_amdgcn_readfirstlane((b - a + TM - 1) / TM);
    if (q < pre + mtiles || e + 1 >= min(E, (owner + 1) * per)) break;
    pre += mtiles;
  }
  e = __builtin_amdgcn_readfirstlane(e);
  a = __builtin_amdgcn_readfirstlane(a);
  b = __builtin_amdgcn_readfirstlane(b);
  pre = __builtin_amdgcn_readfirstlane(pre);
  mtiles = __builtin_amdgcn_readfirstlane(mtiles);
  tile_pair(item - pre * NT, mtiles, NT, mt, nt);
  return true;
}

}  // namespace moe
