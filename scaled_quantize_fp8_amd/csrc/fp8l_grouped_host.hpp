// Host side of the grouped launches (fp8l_grouped.hpp), shared by the FP8
// and the 8-bit integer entry points.
#pragma once

#include <math.h>

#include "fp8l_grouped.hpp"
#include "fp8l_host.hpp"
#include "fp8l_skinny.hpp"

namespace fp8l {

// Most units of `per` rows that T rows in E groups can need: a group with
// rows adds less than one unit to T / per.
inline int64_t most_units(int64_t T, int64_t E, int64_t per) {
  const int64_t live = E < T ? E : T;
  return (T + live * (per - 1)) / per;
}

// Sizes of a grouped call: 32-bit row numbers, also of the rows of a tile or
// of loads in flight that end behind the last row, and tile numbers of every
// tile choice (units of 16 rows by 16 columns at least) below 2^31.
inline int check_grouped(int64_t T, int64_t E, int64_t N, int64_t K) {
  if (T < 0 || T > INT32_MAX - 1024 || E < 1 || E > 65535 || N < 0 || K < 0) return FP8_ERR_SHAPE;
  if (N > INT32_MAX || K > INT32_MAX) return FP8_ERR_SHAPE;
  if (!mul_ok(T, K) || !mul_ok(T, N) || !mul_ok(N, K) || !mul_ok(N * K, E)) return FP8_ERR_SHAPE;
  const int64_t un = (N + 127) / 128, uk = (K + 127) / 128;
  const int64_t u = most_units(T, E, 16);
  if (u * (un > uk ? un : uk) > INT32_MAX / 16) return FP8_ERR_SHAPE;
  if (un * uk > INT32_MAX / 4 || (un * uk + 8) * E > INT32_MAX / 2) return FP8_ERR_SHAPE;
  return FP8_OK;
}

// A launch takes fewer than 2^32 threads.  The general tile, which has the
// fewest per output (256 for 128x128), stands in where a chosen tile's blocks
// would be too many; a call that is too large for it is refused.
inline bool grid_fits(int64_t blocks, int threads) { return blocks + 8 < (1LL << 32) / threads; }
inline bool rows_grid_fits(int64_t T, int64_t E, int64_t N) {
  return grid_fits(most_units(T, E, kBM) * ((N + kBN - 1) / kBN), kGThreads);
}

inline void finish_grouped_args(GemmArgs& g, const GroupStrides& s) {
  g.batch = 1;
  g.a_vec = aligned16(g.a) && g.lda % 16 == 0;
  g.b_vec = aligned16(g.b) && g.ldb % 16 == 0 && s.b % 16 == 0;
  g.c_vec = ((uintptr_t)g.c & 7u) == 0 && g.ldc % 4 == 0 && s.c % 4 == 0;
}

// The pipelined bodies need 16-byte pieces that never straddle a row end and
// byte offsets below 2^31 within what one buffer resource covers: of A the
// rows of one tile, of B one group's matrix.
template <int LB>
bool rows_fast_ok(const GemmArgs& g, const GroupStrides& s) {
  const int64_t b_rows = LB == kKContig ? g.Nc : g.Kc;
  const int64_t b_inner = LB == kKContig ? g.Kc : g.Nc;
  return aligned16(g.a) && aligned16(g.b) && aligned16(g.c) && (!g.bias || aligned16(g.bias)) &&
         g.Nc % 8 == 0 && g.ldc % 8 == 0 && g.lda % 16 == 0 && g.ldb % 16 == 0 &&
         g.Kc % 16 == 0 && b_inner % 16 == 0 && s.b % 16 == 0 && s.bias % 8 == 0 &&
         512 * g.lda < (1LL << 31) && (b_rows + 256) * g.ldb < (1LL << 31);
}

// Waves that split K in a skinny launch of `waves` tile columns, doubled
// while a wave has over 24 pieces of K (16 experts of 4096 -> 11008, one row
// each: 130 us at 32 pieces per wave, 105 at 16), or the chip has room for
// more waves and pieces to give them (one row, 4096 -> 11008: 12.6 us at 8
// waves against 13.6 at 2 and 21.7 at 1; 1536 -> 6912: 5.4 at 4, 6.7 at 8 with
// one or two pieces each), or there are so few waves that any split helps
// (512 -> 512: 3.4 us at 8 waves, 4.5 at 1).
inline int skinny_kw(int64_t waves, int64_t K) {
  const int64_t pieces = (K + 127) / 128;
  int kw = 1;
  while (kw < 8 && (pieces > 24 * kw || (waves * kw < 8192 && pieces >= 4 * kw) ||
                    (waves * kw < 1024 && 2 * pieces > kw)))
    kw *= 2;
  return kw;
}

// Rows of a skinny choice's tiles.
inline int skinny_rows(int tile) {
  switch (tile) {
    case kTileSkinny16: case kTileSkinny16Any: return 16;
    case kTileSkinny32: case kTileSkinny32Any: return 32;
    case kTileSkinny48: return 48;
    default: return 64;
  }
}

// Microseconds of a launch of `tiles` tiles with contraction K, from fits to
// a sweep of the integer GEMM over 64 .. 4096 rows of six layer shapes: a
// fixed part per launch and per round of tiles on the CUs (first stages,
// epilogue), and a part per unit of K.  Measured on a card somewhat faster
// than the sweep's, K = 1536 / 4096 / 11008, against the model:
//   128x128, one block per CU, a full round:  14 / 23 /  49 us (14 / 25 /  55)
//   256x256, a full round:                    35 / 67 / 163    (32 / 64 / 151)
//   256x256, half the CUs:                    29 / 47 / 107    (as a full one)
//   128x256, one block per CU:                25 / 43 / 104    (20 / 41 /  96)
//   128x256, two blocks per CU:               36 / 74 / 196    (47 / 109 / 278)
// The quarter round added to 128x256 stands for uneven last rounds and ragged
// groups; on full rounds it and the slope put the model 23 to 47% too high
// (256 to 2048 tiles more than one per CU), so that tile is taken where it
// wins clearly only.  FP8 and crosswise operands take the same fit.
inline double tile_us(int tile, double tiles, double K) {
  const double cus = cu_count();
  switch (tile) {
    case kTile128x128w8: return 3 + ceil(tiles / cus) * (4 + K * 0.0044);
    case kTile256x256w8: return 3 + ceil(tiles / cus) * (10 + K * 0.0125);
    default: {  // kTile128x256
      if (tiles <= cus) return 8 + K * 0.0080;
      const double rounds = tiles / (2 * cus) + 0.25;
      return 3 + (rounds < 1 ? 1 : rounds) * (5 + K * 0.0195);
    }
  }
}

// The fastest of the three for launches of t128 tiles of 128x128, t12 of
// 128x256, t256 of 256x256.
inline int pick_of(double t128, double t12, double t256, double K, double* us) {
  const double a = tile_us(kTile128x128w8, t128, K), b = tile_us(kTile128x256, t12, K),
               c = tile_us(kTile256x256w8, t256, K);
  *us = a < b ? (a < c ? a : c) : (b < c ? b : c);
  return *us == a ? kTile128x128w8 : (*us == b ? kTile128x256 : kTile256x256w8);
}

// The same for the skinny kernel: a piece of 128 bytes of K for 16 columns
// takes 0.13 us of a CU with up to 16 rows (HBM bound), 0.19 with 32, 0.25
// with 48, 0.32 with 64 (A comes from L2 for every 16 columns); of blocks
// beyond one per CU about a third overlaps.
inline double skinny_us(int mt, double units, int64_t N, int64_t K) {
  const int64_t cols = (N + 15) / 16;
  const int kw = skinny_kw((int64_t)(units * cols), K), jw = 8 / kw;
  const double blocks = units * (double)((cols + jw - 1) / jw);
  const double load = blocks / cu_count();
  const double per_piece[4] = {0.13, 0.19, 0.25, 0.32};
  return 3.5 + (load < 1 ? 1 : 0.3 + 0.7 * load) * (double)((K + 127) / 128) * jw * per_piece[mt - 1];
}

// Units of `per` rows to expect of T rows in E groups of unknown sizes: rows
// thrown at the groups at random hit E (1 - exp(-T / E)) of them, and each of
// those loses half a unit.
inline double expected_units(int64_t T, int64_t E, int64_t per) {
  const double most = (double)most_units(T, E, per);
  if (E == 1) return most;
  const double live = E * (1.0 - exp(-(double)T / E));
  const double u = (double)T / per + 0.5 * live;
  return u < live ? live : (u < most ? u : most);
}

// The fastest tile for T rows in E groups, N columns, contraction K.
inline int pick_tile(int64_t T, int64_t E, int64_t N, int64_t K, bool skinny) {
  const double u128 = expected_units(T, E, 128), u256 = expected_units(T, E, 256);
  const double n128 = (double)((N + 127) / 128), n256 = (double)((N + 255) / 256);
  double us = 0;
  int best = pick_of(u128 * n128, u128 * n256, u256 * n256, (double)K, &us);
  for (int mt = 1; skinny && mt <= 4; ++mt) {
    const double t = skinny_us(mt, expected_units(T, E, 16 * mt), N, K);
    if (t < us) us = t, best = kTileSkinny16 + mt - 1;
  }
  return best;
}

// The same where the pipelined tiles cannot run (odd sizes, unaligned
// pointers): the general tile (two blocks per CU; 2.5 us per 128 of K alone,
// 3.3 for two), or the skinny kernel's form for any alignment, whose pieces
// take 1.6 (64 rows: 2) times as long.  The 64-row form is for many rows of a
// narrow W (8192 x 129 x 4097: 76 us, 83 with 32 rows, 85 on the general tile).
inline int pick_any(int64_t T, int64_t E, int64_t N, int64_t K, bool skinny) {
  const double cus = cu_count(), steps = (double)((K + 127) / 128);
  const double tiles = expected_units(T, E, 128) * (double)((N + 127) / 128);
  double us = 5 + (tiles <= cus ? 2.5 : 3.3 * (tiles / (2 * cus) + 0.5)) * steps;
  int best = kTileV1;
  const int mts[3] = {1, 2, 4}, ids[3] = {kTileSkinny16Any, kTileSkinny32Any, kTileSkinny64Any};
  for (int i = 0; skinny && i < 3; ++i) {
    const double t = (i < 2 ? 1.6 : 2.0) * skinny_us(mts[i], expected_units(T, E, 16 * mts[i]), N, K);
    if (t < us) us = t, best = ids[i];
  }
  return best;
}

// The tile itself, or the general one where its grid would be too large.
inline int tile_that_fits(int tile, int64_t T, int64_t E, int64_t N, int64_t K) {
  int64_t blocks = 0;
  switch (tile) {
    case kTile128x128w8: blocks = most_units(T, E, 128) * ((N + 127) / 128); break;
    case kTile128x256: blocks = most_units(T, E, 128) * ((N + 255) / 256); break;
    case kTile256x256w8: blocks = most_units(T, E, 256) * ((N + 255) / 256); break;
    case kTileV1: return tile;
    default: {  // skinny, of skinny_rows() rows
      const int64_t units = most_units(T, E, skinny_rows(tile)), cols = (N + 15) / 16;
      const int jw = 8 / skinny_kw(units * cols, K);
      blocks = units * ((cols + jw - 1) / jw);
    }
  }
  return grid_fits(blocks, tile == kTile128x256 ? 256 : 512) ? tile : kTileV1;
}

// Tile of a rows launch.
template <int LB>
int rows_tile(const GemmArgs& g, const Groups& gr, const GroupStrides& s) {
  const int f = forced_tile();
  int tile;
  if (!rows_fast_ok<LB>(g, s))
    tile = f == kTileV1 || (LB == kKContig && f >= kTileSkinny16Any) ? f
                        : pick_any(gr.T, gr.E, g.Nc, g.Kc, LB == kKContig);
  else if (f == kTileV1 || f == kTile128x128w8 || f == kTile128x256 || f == kTile256x256w8 ||
           (LB == kKContig && f >= kTileSkinny16))
    tile = f;
  else
    tile = pick_tile(gr.T, gr.E, g.Nc, g.Kc, LB == kKContig);
  return tile_that_fits(tile, gr.T, gr.E, g.Nc, g.Kc);
}

// Tile of a contract launch, by the mean group (4093 rows in 32 groups, dW of
// 4096 x 1024: 82 us on 128x256, 88 on 256x256, 116 on 128x128).
// One resource covers a group's rows of both operands: at most all T rows.
inline bool contract_fast_ok(const GemmArgs& g) {
  return aligned16(g.a) && aligned16(g.b) && aligned16(g.c) && g.lda % 16 == 0 &&
         g.ldb % 16 == 0 && (g.Kc + 256) * g.lda < (1LL << 31) &&
         (g.Kc + 256) * g.ldb < (1LL << 31);
}
// Blocks of one group: its tiles of bm x bn, rounded up to 8.
inline int64_t contract_pad(const GemmArgs& g, int bm, int bn) {
  return ((((g.Mc + bm - 1) / bm) * ((g.Nc + bn - 1) / bn)) + 7) & ~7LL;
}
inline int contract_tile(const GemmArgs& g, const Groups& gr) {
  if (!contract_fast_ok(g)) return kTileV1;
  int tile = forced_tile();
  if (tile == kTileV1) return tile;
  if (tile != kTile128x128w8 && tile != kTile128x256 && tile != kTile256x256w8) {
    const double m128 = (double)((g.Mc + 127) / 128) * gr.E, m256 = (double)((g.Mc + 255) / 256) * gr.E;
    const double n128 = (double)((g.Nc + 127) / 128), n256 = (double)((g.Nc + 255) / 256);
    double us = 0;
    tile = pick_of(m128 * n128, m128 * n256, m256 * n256, (double)gr.T / gr.E, &us);
  }
  const int bm = tile == kTile256x256w8 ? 256 : 128, bn = tile == kTile128x128w8 ? 128 : 256;
  return grid_fits(contract_pad(g, bm, bn) * gr.E, tile == kTile128x256 ? 256 : 512) ? tile : kTileV1;
}

// One tile shape for dX and dW in a shared launch: the smallest sum.
inline int pick_bwd(const GemmArgs& gx, const GemmArgs& gw, const Groups& gr) {
  const int tiles[3] = {kTile128x128w8, kTile128x256, kTile256x256w8};
  const int bm[3] = {128, 128, 256}, bn[3] = {128, 256, 256};
  int best = kTile128x128w8;
  double us = 1e30;
  for (int i = 0; i < 3; ++i) {
    const double x = expected_units(gr.T, gr.E, bm[i]) * (double)((gx.Nc + bn[i] - 1) / bn[i]);
    const double w = (double)((gw.Mc + bm[i] - 1) / bm[i]) * ((gw.Nc + bn[i] - 1) / bn[i]) * gr.E;
    const double t = tile_us(tiles[i], x, (double)gx.Kc) + tile_us(tiles[i], w, (double)gr.T / gr.E);
    if (t < us) us = t, best = tiles[i];
  }
  return best;
}

template <class Tile, bool I8>
void launch_rows_t(GemmArgs& g, const Groups& gr, const GroupStrides& s, const GroupedSide& side,
                   hipStream_t st) {
  static std::atomic<bool> lds_set[64];
  set_lds_limit((const void*)grouped_rows_kernel<Tile, I8>, Tile::kLds, lds_set);
  g.tiles_n = (int32_t)((g.Nc + Tile::kBN - 1) / Tile::kBN);
  const int64_t most = (most_units(gr.T, gr.E, Tile::kBM) * g.tiles_n + 7) & ~7LL;
  hipLaunchKernelGGL((grouped_rows_kernel<Tile, I8>), dim3((unsigned)most), dim3(Tile::kThreads),
                     Tile::kLds, st, g, gr, s, side);
}

template <class S>
void launch_skinny_groups(GemmArgs& g, const Groups& gr, const GroupStrides& s,
                          const GroupedSide& side, hipStream_t st) {
  const int64_t units = most_units(gr.T, gr.E, S::kBM);
  const int64_t cols = (g.Nc + S::kWaveN - 1) / S::kWaveN;
  const int kw = skinny_kw(units * cols, g.Kc), jw = 8 / kw;
  g.tiles_n = (int32_t)((cols + jw - 1) / jw);
  const int64_t most = (units * g.tiles_n + 7) & ~7LL;
  hipLaunchKernelGGL((skinny_groups_kernel<S>), dim3((unsigned)most), dim3(S::kThreads),
                     kw > 1 ? S::kLds : 0, st, g, gr, s, side, kw);
}

template <class S>
void launch_skinny(GemmArgs& g, hipStream_t st) {
  g.tiles_m = (int32_t)((g.Mc + S::kBM - 1) / S::kBM);
  const int64_t cols = (g.Nc + S::kWaveN - 1) / S::kWaveN;
  const int kw = skinny_kw(g.tiles_m * cols, g.Kc), jw = 8 / kw;
  g.tiles_n = (int32_t)((cols + jw - 1) / jw);
  hipLaunchKernelGGL((skinny_kernel<S>), dim3((unsigned)g.tiles_m * (unsigned)g.tiles_n),
                     dim3(S::kThreads), kw > 1 ? S::kLds : 0, st, g, kw);
}

template <int LB, int FA, int FB>
void launch_rows(GemmArgs& g, const Groups& gr, const GroupStrides& s, const GroupedSide& side,
                 int tile, hipStream_t st) {
  if constexpr (LB == kKContig) {
    if (tile == kTileSkinny16Any)
      return launch_skinny_groups<Skinny<FA, FB, 1, true>>(g, gr, s, side, st);
    if (tile == kTileSkinny32Any)
      return launch_skinny_groups<Skinny<FA, FB, 2, true>>(g, gr, s, side, st);
    if (tile == kTileSkinny64Any)
      return launch_skinny_groups<Skinny<FA, FB, 4, true>>(g, gr, s, side, st);
    if (tile == kTileSkinny16) return launch_skinny_groups<Skinny<FA, FB, 1>>(g, gr, s, side, st);
    if (tile == kTileSkinny32) return launch_skinny_groups<Skinny<FA, FB, 2>>(g, gr, s, side, st);
    if (tile == kTileSkinny48) return launch_skinny_groups<Skinny<FA, FB, 3>>(g, gr, s, side, st);
    if (tile == kTileSkinny64) return launch_skinny_groups<Skinny<FA, FB, 4>>(g, gr, s, side, st);
  }
  if (tile == kTile256x256w8)
    launch_rows_t<Tile256<kKContig, LB, FA, FB>, FA == kI8>(g, gr, s, side, st);
  else if (tile == kTile128x256)
    launch_rows_t<Tile128x256<kKContig, LB, FA, FB>, FA == kI8>(g, gr, s, side, st);
  else if (tile == kTile128x128w8)
    launch_rows_t<Tile128<kKContig, LB, FA, FB>, FA == kI8>(g, gr, s, side, st);
  else
    launch_rows_t<TileAny<kKContig, LB, FA, FB>, FA == kI8>(g, gr, s, side, st);
}

// The side work alone, for a call without tiles.
static __global__ __launch_bounds__(64) void grouped_side_kernel(GroupedSide s) { grouped_side(s); }

inline void launch_side(const GroupedSide& s, hipStream_t st) {
  if (s.fold[0].ring || s.fold[1].ring || s.scale_dst[0] || s.scale_dst[1] || s.amax_dst[0] ||
      s.amax_dst[1])
    hipLaunchKernelGGL(grouped_side_kernel, dim3(1), dim3(64), 0, st, s);
}

}  // namespace fp8l
