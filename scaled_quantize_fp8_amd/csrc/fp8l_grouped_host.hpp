// Host side of the grouped launches (fp8l_grouped.hpp), shared by the FP8
// and the 8-bit integer entry points.
#pragma once

#include "fp8l_grouped.hpp"
#include "fp8l_host.hpp"

namespace fp8l {

// Most units of `per` rows that T rows in E groups can need: a group with
// rows adds less than one unit to T / per.
inline int64_t most_units(int64_t T, int64_t E, int64_t per) {
  const int64_t live = E < T ? E : T;
  return (T + live * (per - 1)) / per;
}

// Sizes of a grouped call: 32-bit row offsets, and tile numbers of every
// tile choice below 2^31 (128 is the smallest tile edge).
inline int check_grouped(int64_t T, int64_t E, int64_t N, int64_t K) {
  if (T < 0 || T > INT32_MAX || E < 1 || E > 65535 || N < 0 || K < 0) return FP8_ERR_SHAPE;
  if (N > INT32_MAX || K > INT32_MAX) return FP8_ERR_SHAPE;
  if (!mul_ok(T, K) || !mul_ok(T, N) || !mul_ok(N, K) || !mul_ok(N * K, E)) return FP8_ERR_SHAPE;
  const int64_t un = (N + 127) / 128, uk = (K + 127) / 128;
  const int64_t u = most_units(T, E, 16);
  if (u * (un > uk ? un : uk) > INT32_MAX / 2) return FP8_ERR_SHAPE;
  if (un * uk > INT32_MAX / 4 || (un * uk + 8) * E > INT32_MAX) return FP8_ERR_SHAPE;
  return FP8_OK;
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

// Tile of a rows launch, by the mean group (the host knows no other):
// 256x256 from 96 rows on (8190 rows in 64 groups, 1536 -> 6912: 228 us
// against 303 on 128x128), else 128x128.
template <int LB>
int rows_tile(const GemmArgs& g, const Groups& gr, const GroupStrides& s) {
  if (!rows_fast_ok<LB>(g, s)) return kTileV1;
  const int f = forced_tile();
  if (f == kTileV1 || f == kTile128x128w8 || f == kTile256x256w8) return f;
  return gr.T / gr.E >= 96 ? kTile256x256w8 : kTile128x128w8;
}

// Tile of a contract launch: 256x256 unless dW is small (4096 x 1024 in 32
// groups with the dX of 4093 rows: 171 us against 263 on 128x128).
inline int contract_tile(const GemmArgs& g, const Groups& gr) {
  // one resource covers a group's rows of both operands: at most all T rows
  const bool ok = aligned16(g.a) && aligned16(g.b) && aligned16(g.c) && g.lda % 16 == 0 &&
                  g.ldb % 16 == 0 && (g.Kc + 256) * g.lda < (1LL << 31) &&
                  (g.Kc + 256) * g.ldb < (1LL << 31);
  if (!ok) return kTileV1;
  const int f = forced_tile();
  if (f == kTileV1 || f == kTile128x128w8 || f == kTile256x256w8) return f;
  const int64_t tiles = ((g.Mc + 255) / 256) * ((g.Nc + 255) / 256) * gr.E;
  return 2 * tiles >= cu_count() ? kTile256x256w8 : kTile128x128w8;
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

template <int LB, int FA, int FB>
void launch_rows(GemmArgs& g, const Groups& gr, const GroupStrides& s, const GroupedSide& side,
                 int tile, hipStream_t st) {
  if (tile == kTile256x256w8)
    launch_rows_t<Tile256<kKContig, LB, FA, FB>, FA == kI8>(g, gr, s, side, st);
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
