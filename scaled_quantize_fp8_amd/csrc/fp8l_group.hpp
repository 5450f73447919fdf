// Ragged groups of rows (the experts' linear layers): E groups of
// consecutive rows of a [T, ..] matrix, group e being rows
// [off[e], off[e+1]), off int32 in device memory.  Nothing about the groups
// is known on the host; every block finds its work from off.
//
// A row count is cut into units (a tile's rows, a chunk of a column sum) and
// the units of all groups are numbered group by group.  A wave finds unit u
// with one group per lane: a prefix sum over the lanes' unit counts, then
// the first lane whose sum passes u.  All waves of a block do the same work
// on the same values, so no LDS and no barrier is needed.
//
// Offsets are clamped to [0, T] and each group to start <= end where they
// are read: offsets that decrease or pass T give unspecified results, and
// no access outside the T rows.
#pragma once

#include "fp8l_device.hpp"
#include "fp8l_gemm.hpp"

namespace fp8l {

struct Groups {
  const int32_t* off;  // [E + 1]
  int32_t E;
  int32_t T;
};

struct GroupSpan {
  int32_t e;           // group, or -1 when the unit lies past the last group
  int32_t start, end;  // its rows
  int32_t unit;        // unit's index within the group
  int32_t before;      // units of the groups before it
};

FP8L_DEV int group_edge(const Groups& g, int i) { return min(max(g.off[i], 0), g.T); }

// Inclusive prefix sum over the 64 lanes: shifts inside the rows of 16 lanes
// (a lane without a source adds 0), then each row's total to the later rows.
FP8L_DEV int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);  // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);  // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);  // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15, rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31, rows 2 and 3
  return v;
}

FP8L_DEV int units_of(int rows, int per) { return (rows + per - 1) / per; }

// Units (of `per` rows) over all groups; every lane of the wave calls it.
FP8L_DEV int group_units(const Groups& g, int per) {
  const int lane = threadIdx.x & 63;
  int total = 0;
  for (int e0 = 0; e0 < g.E; e0 += 64) {
    const int e = e0 + lane;
    int n = 0;
    if (e < g.E) {
      const int s = group_edge(g, e);
      n = units_of(max(group_edge(g, e + 1), s) - s, per);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d);
    total += n;
  }
  return __builtin_amdgcn_readfirstlane(total);
}

// The group that holds unit u (uniform over the wave).
FP8L_DEV GroupSpan find_group(const Groups& g, int per, int u) {
  const int lane = threadIdx.x & 63;
  int carry = 0;
  for (int e0 = 0; e0 < g.E; e0 += 64) {
    const int e = e0 + lane;
    int s = 0, t = 0;
    if (e < g.E) {
      s = group_edge(g, e);
      t = max(group_edge(g, e + 1), s);
    }
    const int n = units_of(t - s, per);
    const int incl = carry + wave_scan(n);
    const unsigned long long hit = __ballot(incl > u);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      GroupSpan r;
      r.e = e0 + l;
      r.start = __builtin_amdgcn_readlane(s, l);
      r.end = __builtin_amdgcn_readlane(t, l);
      r.before = __builtin_amdgcn_readlane(incl - n, l);
      r.unit = u - r.before;
      return r;
    }
    carry = __builtin_amdgcn_readlane(incl, 63);
  }
  return GroupSpan{-1, 0, 0, 0, carry};
}

// This block's tile of a launch over all groups' units times tiles_n tile
// columns (e = -1: none): tiles numbered group by group, XCD x (blocks
// x mod 8) taking the x-th eighth; tm within the group.  With at most 64
// groups one pass over the offsets does it.
FP8L_DEV GroupSpan rows_work(const Groups& g, int per, int tiles_n, int& tm, int& tn) {
  const int lane = threadIdx.x & 63;
  const int x = blockIdx.x % 8, k = blockIdx.x / 8;
  int s = 0, t = 0, n = 0, incl = 0, total;
  if (g.E <= 64) {
    if (lane < g.E) {
      s = group_edge(g, lane);
      t = max(group_edge(g, lane + 1), s);
      n = units_of(t - s, per);
    }
    incl = wave_scan(n);
    total = __builtin_amdgcn_readlane(incl, 63);
  } else {
    total = group_units(g, per);
  }
  const int nb = total * tiles_n, q = nb / 8, r = nb % 8;
  if (k >= q + (x < r ? 1 : 0)) return GroupSpan{-1, 0, 0, 0, 0};
  const int pid = x * q + min(x, r) + k;
  const int u = pid / tiles_n;
  GroupSpan sp;
  if (g.E <= 64) {
    const unsigned long long hit = __ballot(incl > u);
    if (!hit) return GroupSpan{-1, 0, 0, 0, 0};
    const int l = __builtin_ctzll(hit);
    sp.e = l;
    sp.start = __builtin_amdgcn_readlane(s, l);
    sp.end = __builtin_amdgcn_readlane(t, l);
    sp.before = __builtin_amdgcn_readlane(incl - n, l);
    sp.unit = u - sp.before;
  } else {
    sp = find_group(g, per, u);
    if (sp.e < 0) return sp;
  }
  tile_coords(pid - sp.before * tiles_n, units_of(sp.end - sp.start, per), tiles_n, tm, tn);
  return sp;
}

// Rows and units of group e itself, and the units before it.
FP8L_DEV GroupSpan group_span(const Groups& g, int per, int e_) {
  const int lane = threadIdx.x & 63;
  GroupSpan r = {e_, 0, 0, 0, 0};
  for (int e0 = 0; e0 < e_; e0 += 64) {
    const int e = e0 + lane;
    int n = 0;
    if (e < e_) {
      const int s = group_edge(g, e);
      n = units_of(max(group_edge(g, e + 1), s) - s, per);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d);
    r.before += n;
  }
  r.before = __builtin_amdgcn_readfirstlane(r.before);
  r.start = __builtin_amdgcn_readfirstlane(group_edge(g, e_));
  r.end = max(__builtin_amdgcn_readfirstlane(group_edge(g, e_ + 1)), r.start);
  return r;
}

}  // namespace fp8l
