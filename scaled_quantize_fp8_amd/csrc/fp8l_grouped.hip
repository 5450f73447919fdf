// C entry points of the FP8 linear layers over ragged groups of rows (the
// experts of a mixture).  As in fp8l_api.hip, every check runs before the
// first launch, nothing is allocated and the host never waits.
#include <type_traits>

#include "fp8l_grouped.hpp"
#include "fp8l_grouped_host.hpp"
#include "fp8l_host.hpp"

namespace fp8l {
namespace {

__global__ __launch_bounds__(256) void grouped_db_kernel(DbArgs a, Groups gr) {
  __shared__ float sh[kDbLds / 4];
  db_block(a, gr, blockIdx.x, sh);
}

int64_t db_blocks(const DbArgs& a, const Groups& gr) {
  const int width = a.ws ? 64 : 256;
  return a.db ? (a.N + width - 1) / width * gr.E : 0;
}

template <class Tile>
void launch_contract(GemmArgs& g, const Groups& gr, const GroupStrides& s, hipStream_t st) {
  static std::atomic<bool> lds_set[64];
  set_lds_limit((const void*)grouped_contract_kernel<Tile>, Tile::kLds, lds_set);
  g.tiles_m = (int32_t)((g.Mc + Tile::kBM - 1) / Tile::kBM);
  g.tiles_n = (int32_t)((g.Nc + Tile::kBN - 1) / Tile::kBN);
  const int pad = (int)contract_pad(g, Tile::kBM, Tile::kBN);
  hipLaunchKernelGGL((grouped_contract_kernel<Tile>), dim3((unsigned)gr.E * (unsigned)pad),
                     dim3(Tile::kThreads), Tile::kLds, st, g, gr, s, pad);
}

// Calls f(integral_constant fa, integral_constant fb) for two FP8 formats.
template <class F>
void by_formats(int fa, int fb, F&& f) {
  using E4 = std::integral_constant<int, kE4M3>;
  using E5 = std::integral_constant<int, kE5M2>;
  if (fa == kE4M3 && fb == kE4M3) f(E4{}, E4{});
  else if (fa == kE4M3) f(E4{}, E5{});
  else if (fb == kE4M3) f(E5{}, E4{});
  else f(E5{}, E5{});
}

// dX: A = G8 rows, B = W8[e] [N, K] read crosswise.
void launch_dx(GemmArgs& g, int fa, int fb, const Groups& gr, const GroupStrides& s,
               const GroupedSide& side, hipStream_t st) {
  const int tile = rows_tile<kCross>(g, gr, s);
  by_formats(fa, fb, [&](auto a, auto b) {
    constexpr int FA = decltype(a)::value, FB = decltype(b)::value;
    launch_rows<kCross, FA, FB>(g, gr, s, side, tile, st);
  });
}

// dW: both crosswise.
void launch_dw(GemmArgs& g, int fa, int fb, const Groups& gr, const GroupStrides& s,
               hipStream_t st) {
  const int tile = contract_tile(g, gr);
  by_formats(fa, fb, [&](auto a, auto b) {
    constexpr int FA = decltype(a)::value, FB = decltype(b)::value;
    if (tile == kTile256x256w8)
      launch_contract<Tile256<kCross, kCross, FA, FB>>(g, gr, s, st);
    else if (tile == kTile128x256)
      launch_contract<Tile128x256<kCross, kCross, FA, FB>>(g, gr, s, st);
    else if (tile == kTile128x128w8)
      launch_contract<Tile128<kCross, kCross, FA, FB>>(g, gr, s, st);
    else
      launch_contract<TileAny<kCross, kCross, FA, FB>>(g, gr, s, st);
  });
}

// Blocks of the quantize with column sums; the rows before the first group
// are one more group.
int64_t groupsum_blocks(int64_t T, int64_t E, int64_t N) {
  return most_units(T, E + 1, kColRowsPerChunk) * ((N + kColStrip - 1) / kColStrip);
}

// The quantize of G with the groups' column sums in the same pass; scale
// modes as enqueue_quant (fp8l_api.hip).  Returns whether the fold of the
// ring was left to the caller's next GEMM.
bool enqueue_groupsum(const fp8_operand_t& x, int64_t T, int64_t N, int32_t fmt, uint8_t* q,
                      fp8_ring_t* ring, float* scale_used, float* amax_out, float* ws,
                      const Groups& gr, const RowLimit& limit, hipStream_t st) {
  const bool defer = can_defer(ring);
  const int64_t n = T * N;
  QArgs a = {};
  a.x = x.data;
  a.q = q;
  a.n = n;
  a.rows = T;
  a.cols = N;
  a.scale_used = scale_used;
  a.amax_out = amax_out;
  a.colsum = ws;
  a.vec_ok = aligned16(x.data) && aligned16(q) && N % 8 == 0;
  if (ring) {
    a.ring = reinterpret_cast<RingHdr*>(ring->dev);
    a.hist = reinterpret_cast<float*>(reinterpret_cast<char*>(ring->dev) + sizeof(RingHdr));
    a.hist_len = ring->hist_len;
  }
  a.limit = limit;
  const bool local = !ring && n <= kLocalMost;
  if (!local && (!ring || !ring->seeded)) enqueue_amax(x.data, x.dtype, n, ring, amax_out, limit, st);
  const int strips = (int)((N + kColStrip - 1) / kColStrip);
  const int most = (int)most_units(T, gr.E, kColRowsPerChunk);
  const dim3 grid((unsigned)groupsum_blocks(T, gr.E, N));
  auto run = [&](auto in, auto f, auto mode) {
    hipLaunchKernelGGL((quantize_groupsum_kernel<decltype(in)::value, decltype(f)::value,
                                                 decltype(mode)::value>),
                       grid, dim3(kQThreads), 0, st, a, gr, strips, most);
  };
  auto by_mode = [&](auto in, auto f) {
    if (local) run(in, f, std::integral_constant<int, kScaleLocal>{});
    else if (!ring) run(in, f, std::integral_constant<int, kScaleDyn>{});
    else if (!ring->seeded) run(in, f, std::integral_constant<int, kScaleSeed>{});
    else if (defer) run(in, f, std::integral_constant<int, kScaleDefer>{});
    else run(in, f, std::integral_constant<int, kScaleRing>{});
  };
  auto by_fmt = [&](auto in) {
    if (fmt == FP8_E4M3) by_mode(in, std::integral_constant<int, kE4M3>{});
    else by_mode(in, std::integral_constant<int, kE5M2>{});
  };
  if (x.dtype == FP8_DT_F32) by_fmt(std::integral_constant<int, kInF32>{});
  else if (x.dtype == FP8_DT_F16) by_fmt(std::integral_constant<int, kInF16>{});
  else by_fmt(std::integral_constant<int, kInBF16>{});
  if (ring) ring->seeded = 1;
  return defer;
}

// dX, dW and db in one launch with one tile shape, where both GEMMs can take
// a pipelined tile and the grid takes all three; false: the caller launches
// them one by one.
template <class TX, class TW>
bool launch_bwd_t(GemmArgs& gx, GemmArgs& gw, const Groups& gr, const GroupStrides& sx,
                  const GroupStrides& sw, const GroupedSide& side, const DbArgs& db,
                  hipStream_t st) {
  gx.tiles_n = (int32_t)((gx.Nc + TX::kBN - 1) / TX::kBN);
  gw.tiles_m = (int32_t)((gw.Mc + TW::kBM - 1) / TW::kBM);
  gw.tiles_n = (int32_t)((gw.Nc + TW::kBN - 1) / TW::kBN);
  const int64_t nx = (most_units(gr.T, gr.E, TX::kBM) * gx.tiles_n + 7) & ~7LL;
  const int64_t pad = contract_pad(gw, TW::kBM, TW::kBN);
  const int64_t nw = pad * gr.E, blocks = nx + nw + db_blocks(db, gr);
  if (!grid_fits(blocks, TX::kThreads)) return false;
  static std::atomic<bool> lds_set[64];
  set_lds_limit((const void*)grouped_bwd_kernel<TX, TW>, TX::kLds, lds_set);
  hipLaunchKernelGGL((grouped_bwd_kernel<TX, TW>), dim3((unsigned)blocks), dim3(TX::kThreads),
                     TX::kLds, st, gx, gw, gr, sx, sw, side, (int)nx, (int)nw, (int)pad, db);
  return true;
}

bool launch_bwd(GemmArgs& gx, GemmArgs& gw, int fg, int fw, const Groups& gr,
                const GroupStrides& sx, const GroupStrides& sw, const GroupedSide& side,
                const DbArgs& db, hipStream_t st) {
  if (!rows_fast_ok<kCross>(gx, sx) || !contract_fast_ok(gw)) return false;
  int tile = forced_tile();
  if (tile == kTileV1) return false;
  if (tile != kTile128x128w8 && tile != kTile128x256 && tile != kTile256x256w8)
    tile = pick_bwd(gx, gw, gr);
  bool done = false;
  by_formats(fg, fw, [&](auto a, auto b) {
    constexpr int FG = decltype(a)::value, FW = decltype(b)::value;
    if (tile == kTile128x128w8)
      done = launch_bwd_t<Tile128<kKContig, kCross, FG, FW>, Tile128<kCross, kCross, FG, FW>>(
          gx, gw, gr, sx, sw, side, db, st);
    else if (tile == kTile128x256)
      done = launch_bwd_t<Tile128x256<kKContig, kCross, FG, FW>, Tile128x256<kCross, kCross, FG, FW>>(
          gx, gw, gr, sx, sw, side, db, st);
    else
      done = launch_bwd_t<Tile256<kKContig, kCross, FG, FW>, Tile256<kCross, kCross, FG, FW>>(
          gx, gw, gr, sx, sw, side, db, st);
  });
  return done;
}

}  // namespace
}  // namespace fp8l

using namespace fp8l;

extern "C" {

size_t fp8_grouped_db_workspace_bytes(int64_t T, int32_t E, int64_t N) {
  if (T < 0 || T > INT32_MAX || E < 0 || N < 0) return 0;
  const int64_t units = most_units(T, E, kColRowsPerChunk);
  return mul_ok(units, N) ? (size_t)(4 * units * N) : 0;
}

int fp8_grouped_linear_fwd(int64_t T, int32_t E, int64_t N, int64_t K, const int32_t* offsets,
                           fp8_operand_t x, fp8_operand_t w, int32_t w_scales, const void* bias,
                           int32_t fmt, fp8_ring_t* ring_x, fp8_ring_t* ring_w, void* y,
                           uint8_t* x8_out, uint8_t* w8_out, float* sx_used, float* sw_used,
                           float* amax_x, float* amax_w, hipStream_t stream) {
  int st = check_grouped(T, E, N, K);
  if (st) return st;
  if (!rows_grid_fits(T, E, N)) return FP8_ERR_SHAPE;
  if (!valid_fmt(fmt)) return FP8_ERR_DTYPE;
  if (!offsets) return FP8_ERR_NULL;
  const int32_t f8dt = fmt_dtype(fmt);
  if (is_hp(x.dtype)) {
    if ((st = check_quant(x.data, x.dtype, T * K, fmt, x8_out, ring_x, sx_used, amax_x, stream)))
      return st;
  } else if (x.dtype == f8dt) {
    if ((T * K > 0 && !x.data) || !x.scale) return FP8_ERR_NULL;
  } else {
    return FP8_ERR_DTYPE;
  }
  if (is_hp(w.dtype)) {
    if ((st = check_quant(w.data, w.dtype, E * N * K, fmt, w8_out, ring_w, sw_used, amax_w, stream)))
      return st;
  } else if (w.dtype == f8dt) {
    if (w_scales != 1 && w_scales != E) return FP8_ERR_SHAPE;
    if ((N * K > 0 && !w.data) || !w.scale) return FP8_ERR_NULL;
  } else {
    return FP8_ERR_DTYPE;
  }
  if (ring_x && ring_x == ring_w) return FP8_ERR_RING;
  if (T * N > 0 && !y) return FP8_ERR_NULL;

  const Groups gr = {offsets, E, (int32_t)T};
  GroupedSide side = {};
  GemmArgs g = {};
  GroupStrides s = {};
  if (is_hp(x.dtype)) {
    const RowLimit limit = {offsets + E, T, K};
    if (enqueue_quant(x.data, x.dtype, T * K, fmt, x8_out, ring_x, sx_used, amax_x, nullptr, stream,
                      T * N > 0, limit))
      side.fold[0] = fold_of(ring_x, fmt, amax_x);
    g.a = x8_out;
    g.scale_a = sx_used;
  } else {
    g.a = reinterpret_cast<const uint8_t*>(x.data);
    g.scale_a = x.scale;
    side.scale_src[0] = x.scale;
    side.scale_dst[0] = sx_used;
    side.amax_dst[0] = amax_x;
    side.n[0] = 1;
  }
  if (is_hp(w.dtype)) {
    if (enqueue_quant(w.data, w.dtype, E * N * K, fmt, w8_out, ring_w, sw_used, amax_w, nullptr,
                      stream, T * N > 0))
      side.fold[1] = fold_of(ring_w, fmt, amax_w);
    g.b = w8_out;
    g.scale_b = sw_used;
  } else {
    g.b = reinterpret_cast<const uint8_t*>(w.data);
    g.scale_b = w.scale;
    s.sb = w_scales == E && E > 1 ? 1 : 0;
    side.scale_src[1] = w.scale;
    side.scale_dst[1] = sw_used;
    side.amax_dst[1] = amax_w;
    side.n[1] = w_scales;
  }
  g.lda = K;
  g.ldb = K;
  g.Mc = T;
  g.Nc = N;
  g.Kc = K;
  g.c = reinterpret_cast<uint16_t*>(y);
  g.ldc = N;
  g.bias = bias;
  g.bias_kind = bias ? kBiasBF16 : kBiasNone;
  s.b = N * K;
  s.bias = (int32_t)N;
  finish_grouped_args(g, s);
  if (T * N > 0) {
    const int tile = rows_tile<kKContig>(g, gr, s);
    if (fmt == FP8_E4M3) launch_rows<kKContig, kE4M3, kE4M3>(g, gr, s, side, tile, stream);
    else launch_rows<kKContig, kE5M2, kE5M2>(g, gr, s, side, tile, stream);
  } else {
    launch_side(side, stream);
  }
  return hip_status();
}

int fp8_grouped_linear_bwd(int64_t T, int32_t E, int64_t N, int64_t K, const int32_t* offsets,
                           fp8_operand_t g, int32_t fmt_g, fp8_ring_t* ring_g, fp8_operand_t x8,
                           fp8_operand_t w8, int32_t w_scales, void* dx, void* dw, void* db,
                           float* db_ws, uint8_t* g8_out, float* sg_used, float* amax_g,
                           hipStream_t stream) {
  int st = check_grouped(T, E, N, K);
  if (st) return st;
  if (!valid_fmt(fmt_g)) return FP8_ERR_DTYPE;
  if (!offsets) return FP8_ERR_NULL;
  const bool hp = is_hp(g.dtype);
  if (hp) {
    if ((st = check_quant(g.data, g.dtype, T * N, fmt_g, g8_out, ring_g, sg_used, amax_g, stream)))
      return st;
  } else if (g.dtype == fmt_dtype(fmt_g)) {
    if ((T * N > 0 && !g.data) || !g.scale) return FP8_ERR_NULL;
  } else {
    return FP8_ERR_DTYPE;
  }
  if (dx) {
    if (!is_f8(w8.dtype)) return FP8_ERR_DTYPE;
    if (w_scales != 1 && w_scales != E) return FP8_ERR_SHAPE;
    if ((N * K > 0 && !w8.data) || !w8.scale) return FP8_ERR_NULL;
  }
  if (dw) {
    if (!is_f8(x8.dtype)) return FP8_ERR_DTYPE;
    if ((T * K > 0 && !x8.data) || !x8.scale) return FP8_ERR_NULL;
  }
  const bool sums = hp && db && T > 0 && N > 0;
  if (sums && !db_ws) return FP8_ERR_NULL;
  if (sums && !fp8_grouped_db_workspace_bytes(T, E, N)) return FP8_ERR_SHAPE;

  const Groups gr = {offsets, E, (int32_t)T};
  const uint8_t* g8;
  const float* sg;
  GroupedSide side = {};
  const bool have_dx = dx && T * K > 0, have_dw = dw && N * K > 0;
  DbArgs da = {};
  if (db && N > 0) {
    da.db = reinterpret_cast<uint16_t*>(db);
    da.N = N;
    da.ws = sums ? db_ws : nullptr;
  }
  // every launch below must fit its grid (see grid_fits)
  if ((have_dx && !rows_grid_fits(T, E, K)) || !grid_fits(db_blocks(da, gr), 256) ||
      (have_dw && !grid_fits((((N + kBM - 1) / kBM) * ((K + kBN - 1) / kBN) + 7) * E, kGThreads)) ||
      (sums && !grid_fits(groupsum_blocks(T, E, N), kQThreads)))
    return FP8_ERR_SHAPE;
  if (hp) {
    const RowLimit limit = {offsets + E, T, N};
    bool fold = false;
    if (sums) {
      fold = enqueue_groupsum(g, T, N, fmt_g, g8_out, ring_g, sg_used, amax_g, db_ws, gr, limit,
                              stream);
    } else {
      fold = enqueue_quant(g.data, g.dtype, T * N, fmt_g, g8_out, ring_g, sg_used, amax_g, nullptr,
                           stream, have_dx, limit);
    }
    if (fold) side.fold[0] = fold_of(ring_g, fmt_g, amax_g);
    g8 = g8_out;
    sg = sg_used;
    da.most = (int32_t)most_units(T, E, kColRowsPerChunk);
  } else {
    g8 = reinterpret_cast<const uint8_t*>(g.data);
    sg = g.scale;
    side.scale_src[0] = g.scale;
    side.scale_dst[0] = sg_used;
    side.amax_dst[0] = amax_g;
    side.n[0] = 1;
    da.g8 = g8;
    da.g8_e5m2 = fmt_g == FP8_E5M2;
    da.vec = aligned16(g8) && N % 16 == 0;
    da.scale = sg;
  }
  GemmArgs gx = {}, gw = {};
  GroupStrides sx = {}, sw = {};
  gx.a = g8;
  gx.lda = N;
  gx.b = reinterpret_cast<const uint8_t*>(w8.data);
  gx.ldb = K;
  gx.Mc = T;
  gx.Nc = K;
  gx.Kc = N;
  gx.c = reinterpret_cast<uint16_t*>(dx);
  gx.ldc = K;
  gx.scale_a = sg;
  gx.scale_b = w8.scale;
  sx.b = N * K;
  sx.sb = w_scales == E && E > 1 ? 1 : 0;
  finish_grouped_args(gx, sx);
  gw.a = g8;
  gw.lda = N;
  gw.b = reinterpret_cast<const uint8_t*>(x8.data);
  gw.ldb = K;
  gw.Mc = N;
  gw.Nc = K;
  gw.Kc = T;
  gw.c = reinterpret_cast<uint16_t*>(dw);
  gw.ldc = K;
  gw.scale_a = sg;
  gw.scale_b = x8.scale;
  sw.c = N * K;
  finish_grouped_args(gw, sw);
  if (have_dx && have_dw && w8.dtype == x8.dtype &&
      launch_bwd(gx, gw, fmt_g, dtype_fmt(w8.dtype), gr, sx, sw, side, da, stream))
    return hip_status();
  if (have_dx) launch_dx(gx, fmt_g, dtype_fmt(w8.dtype), gr, sx, side, stream);
  else launch_side(side, stream);
  if (have_dw) launch_dw(gw, fmt_g, dtype_fmt(x8.dtype), gr, sw, stream);
  if (da.db)
    hipLaunchKernelGGL(grouped_db_kernel, dim3((unsigned)db_blocks(da, gr)), dim3(256), 0, stream,
                       da, gr);
  return hip_status();
}

}  // extern "C"
