// C entry points of the linear layers in 8-bit integers with one scale per
// token and one per output channel, dense and over ragged groups of rows.
// Checks run before the first launch; nothing is allocated.
#include <type_traits>

#include "fp8l_grouped_host.hpp"
#include "fp8l_i8.hpp"

namespace fp8l {
namespace {

// One tile per block in XCD-major order; A is moved to the tile's rows, so
// that one buffer resource covers them however many rows there are.
template <class Tile>
__global__ __launch_bounds__(Tile::kThreads, Tile::kBlocks) void i8_gemm_kernel(GemmArgs g) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_i8[];
  int tm, tn;
  tile_coords_xcd(blockIdx.x, g.tiles_m, g.tiles_n, tm, tn);
  const int64_t row = (int64_t)tm * Tile::kBM;
  g.a += row * g.lda;
  g.c += row * g.ldc;
  g.scale_a += row;
  g.Mc = min<int64_t>(g.Mc - row, Tile::kBM);
  Tile::run(g, 0, tn, smem_i8);
}

template <class Tile>
void launch_i8_t(GemmArgs& g, hipStream_t st) {
  static std::atomic<bool> lds_set[64];
  set_lds_limit((const void*)i8_gemm_kernel<Tile>, Tile::kLds, lds_set);
  g.tiles_m = (int32_t)((g.Mc + Tile::kBM - 1) / Tile::kBM);
  g.tiles_n = (int32_t)((g.Nc + Tile::kBN - 1) / Tile::kBN);
  hipLaunchKernelGGL((i8_gemm_kernel<Tile>), dim3((unsigned)g.tiles_m * (unsigned)g.tiles_n),
                     dim3(Tile::kThreads), Tile::kLds, st, g);
}

int i8_tile(const GemmArgs& g) {
  const int f = forced_tile();
  int tile;
  if (!rows_fast_ok<kKContig>(g, GroupStrides{}))
    tile = f == kTileV1 || f >= kTileSkinny16Any ? f : pick_any(g.Mc, 1, g.Nc, g.Kc, true);
  else
    tile = f == kTileV1 || f >= kTile256x256w8 ? f : pick_tile(g.Mc, 1, g.Nc, g.Kc, true);
  return tile_that_fits(tile, g.Mc, 1, g.Nc, g.Kc);
}

// Calls f(integral_constant) for a high-precision input type.
template <class F>
void by_input(int32_t dt, F&& f) {
  if (dt == FP8_DT_F32) f(std::integral_constant<int, kInF32>{});
  else if (dt == FP8_DT_F16) f(std::integral_constant<int, kInF16>{});
  else f(std::integral_constant<int, kInBF16>{});
}

void enqueue_rows(const void* x, int32_t dt, int64_t rows, int64_t cols, int8_t* q, float* scale,
                  const int32_t* valid, hipStream_t st) {
  if (rows == 0) return;
  RowsArgs a = {x, q, scale, rows, cols, 0, valid};
  a.vec_ok = aligned16(x) && ((uintptr_t)q & 7u) == 0 && cols % 8 == 0;
  const int64_t cap = (int64_t)cu_count() * 8;
  const dim3 grid((unsigned)(rows < cap ? rows : cap));
  const bool wide = rows <= 2 * cu_count() && cols >= 4096;
  by_input(dt, [&](auto in) {
    constexpr int IN = decltype(in)::value;
    if (wide)
      hipLaunchKernelGGL((quantize_rows_kernel<IN, 1024>), grid, dim3(1024), 0, st, a);
    else
      hipLaunchKernelGGL((quantize_rows_kernel<IN, kQThreads>), grid, dim3(kQThreads), 0, st, a);
  });
}

// Whether a call's blocks quantize its X themselves (SkinnyFused): the X that
// every 16 columns read again must stay small beside their rows of W, and
// its codes must fit the LDS of two blocks per CU.  Dense: up to 4 rows (one
// token, 4096 -> 11008: 12.0 us against 14.4).  Groups: two rows per expert on
// average (any unit may have 16), unless reading the weights takes so long
// that a launch does not count (16 experts of 45 MB: 108 us against 105).
// groups 0: dense.
bool fuse_rows(const GemmArgs& g, const fp8_operand_t& x, int64_t rows, int64_t groups) {
  if (!is_hp(x.dtype) || !aligned16(x.data) || forced_tile() != kTileAuto) return false;
  if (g.Kc % 16 != 0 || g.Kc < 16 || ((uintptr_t)g.a & 7u) != 0) return false;
  if (!rows_fast_ok<kKContig>(g, GroupStrides{})) return false;
  if (groups == 0) return rows <= 4 && g.Kc <= 16384;
  const int64_t live = rows < groups ? rows : groups;
  return rows <= 2 * groups && g.Kc <= 4096 && live * g.Nc * g.Kc <= (256LL << 20);
}

template <int IN>
void launch_fused(GemmArgs& g, const FusedX& fx, const Groups* gr, const GroupStrides& s,
                  hipStream_t st) {
  using F = SkinnyFused<IN>;
  const int64_t units = gr ? most_units(gr->T, gr->E, 16) : 1, cols = (g.Nc + 15) / 16;
  const int kw = skinny_kw(units * cols, g.Kc), jw = 8 / kw;
  g.tiles_n = (int32_t)((cols + jw - 1) / jw);
  static std::atomic<bool> set_dense[64], set_groups[64];
  if (gr) {
    const int lds = F::lds(16, g.Kc);
    set_lds_limit((const void*)skinny_fused_groups_kernel<IN>, F::lds(16, 4096), set_groups);
    const int64_t most = (units * g.tiles_n + 7) & ~7LL;
    hipLaunchKernelGGL((skinny_fused_groups_kernel<IN>), dim3((unsigned)most), dim3(512), lds, st,
                       g, *gr, s, fx, kw);
  } else {
    set_lds_limit((const void*)skinny_fused_kernel<IN>, F::lds(4, 16384), set_dense);
    hipLaunchKernelGGL((skinny_fused_kernel<IN>), dim3((unsigned)g.tiles_n), dim3(512),
                       F::lds((int)g.Mc, g.Kc), st, g, fx, kw);
  }
}

// 128 * 128 * K stays below 2^31: the int32 sums cannot overflow, whatever
// the codes.
constexpr int64_t kI8MaxK = 131071;

int check_i8(int64_t M, int64_t N, int64_t K, const fp8_operand_t& x, const fp8_operand_t& w,
             int32_t out_dtype, const void* y, const int8_t* x8_out, const float* sx_out) {
  if (K > kI8MaxK) return FP8_ERR_SHAPE;
  if (out_dtype != FP8_DT_BF16 && out_dtype != FP8_DT_F16) return FP8_ERR_DTYPE;
  if (w.dtype != FP8_DT_I8) return FP8_ERR_DTYPE;
  if (is_hp(x.dtype)) {
    if (M * K > 0 && (!x.data || !x8_out)) return FP8_ERR_NULL;
    if (M > 0 && !sx_out) return FP8_ERR_NULL;
  } else if (x.dtype == FP8_DT_I8) {
    if ((M * K > 0 && !x.data) || (M > 0 && !x.scale)) return FP8_ERR_NULL;
  } else {
    return FP8_ERR_DTYPE;
  }
  if ((N * K > 0 && !w.data) || (N > 0 && !w.scale)) return FP8_ERR_NULL;
  if (M * N > 0 && !y) return FP8_ERR_NULL;
  return FP8_OK;
}

// The GEMM's arguments; a high-precision x is yet to be quantized into x8_out.
GemmArgs i8_args(int64_t M, int64_t N, int64_t K, const fp8_operand_t& x, const fp8_operand_t& w,
                 const void* bias, int32_t out_dtype, void* y, int8_t* x8_out, float* sx_out) {
  GemmArgs g = {};
  if (is_hp(x.dtype)) {
    g.a = reinterpret_cast<const uint8_t*>(x8_out);
    g.scale_a = sx_out;
  } else {
    g.a = reinterpret_cast<const uint8_t*>(x.data);
    g.scale_a = x.scale;
  }
  g.lda = K;
  g.b = reinterpret_cast<const uint8_t*>(w.data);
  g.ldb = K;
  g.scale_b = w.scale;
  g.Mc = M;
  g.Nc = N;
  g.Kc = K;
  g.c = reinterpret_cast<uint16_t*>(y);
  g.ldc = N;
  g.bias = bias;
  g.bias_kind = bias ? kBiasBF16 : kBiasNone;  // two bytes each, in y's type
  g.out_f16 = out_dtype == FP8_DT_F16;
  return g;
}

}  // namespace
}  // namespace fp8l

using namespace fp8l;

extern "C" {

int fp8_i8_quantize_rows(const void* x, int32_t in_dtype, int64_t rows, int64_t cols, int8_t* q,
                         float* scale, hipStream_t stream) {
  if (rows < 0 || cols < 0 || !mul_ok(rows, cols)) return FP8_ERR_SHAPE;
  if (!is_hp(in_dtype)) return FP8_ERR_DTYPE;
  if (rows * cols > 0 && (!x || !q)) return FP8_ERR_NULL;
  if (rows > 0 && !scale) return FP8_ERR_NULL;
  enqueue_rows(x, in_dtype, rows, cols, q, scale, nullptr, stream);
  return hip_status();
}

int fp8_i8_linear_fwd(int64_t M, int64_t N, int64_t K, fp8_operand_t x, fp8_operand_t w,
                      const void* bias, int32_t out_dtype, void* y, int8_t* x8_out, float* sx_out,
                      hipStream_t stream) {
  if (M < 0 || N < 0 || K < 0) return FP8_ERR_SHAPE;
  if (!mul_ok(M, K) || !mul_ok(N, K) || !mul_ok(M, N)) return FP8_ERR_SHAPE;
  if (((M + 127) / 128) > INT32_MAX / ((N + 127) / 128 + 1) || !rows_grid_fits(M, 1, N))
    return FP8_ERR_SHAPE;
  const int st = check_i8(M, N, K, x, w, out_dtype, y, x8_out, sx_out);
  if (st) return st;
  GemmArgs g = i8_args(M, N, K, x, w, bias, out_dtype, y, x8_out, sx_out);
  finish_grouped_args(g, GroupStrides{});
  if (M > 0 && N > 0 && fuse_rows(g, x, M, 0)) {
    by_input(x.dtype, [&](auto in) {
      launch_fused<decltype(in)::value>(g, FusedX{x.data, x8_out, sx_out}, nullptr, GroupStrides{},
                                        stream);
    });
    return hip_status();
  }
  if (is_hp(x.dtype)) enqueue_rows(x.data, x.dtype, M, K, x8_out, sx_out, nullptr, stream);
  if (M > 0 && N > 0) {
    const int tile = i8_tile(g);
    if (tile == kTileSkinny16Any) launch_skinny<Skinny<kI8, kI8, 1, true>>(g, stream);
    else if (tile == kTileSkinny32Any) launch_skinny<Skinny<kI8, kI8, 2, true>>(g, stream);
    else if (tile == kTileSkinny64Any) launch_skinny<Skinny<kI8, kI8, 4, true>>(g, stream);
    else if (tile == kTileSkinny16) launch_skinny<Skinny<kI8, kI8, 1>>(g, stream);
    else if (tile == kTileSkinny32) launch_skinny<Skinny<kI8, kI8, 2>>(g, stream);
    else if (tile == kTileSkinny48) launch_skinny<Skinny<kI8, kI8, 3>>(g, stream);
    else if (tile == kTileSkinny64) launch_skinny<Skinny<kI8, kI8, 4>>(g, stream);
    else if (tile == kTile128x256) launch_i8_t<Tile128x256<kKContig, kKContig, kI8, kI8>>(g, stream);
    else if (tile == kTile256x256w8) launch_i8_t<Tile256<kKContig, kKContig, kI8, kI8>>(g, stream);
    else if (tile == kTile128x128w8) launch_i8_t<Tile128<kKContig, kKContig, kI8, kI8>>(g, stream);
    else launch_i8_t<TileAny<kKContig, kKContig, kI8, kI8>>(g, stream);
  }
  return hip_status();
}

int fp8_i8_grouped_linear_fwd(int64_t T, int32_t E, int64_t N, int64_t K, const int32_t* offsets,
                              fp8_operand_t x, fp8_operand_t w, const void* bias,
                              int32_t out_dtype, void* y, int8_t* x8_out, float* sx_out,
                              hipStream_t stream) {
  int st = check_grouped(T, E, N, K);
  if (st) return st;
  if (!rows_grid_fits(T, E, N)) return FP8_ERR_SHAPE;
  if (!offsets) return FP8_ERR_NULL;
  if ((st = check_i8(T, N, K, x, w, out_dtype, y, x8_out, sx_out))) return st;
  GemmArgs g = i8_args(T, N, K, x, w, bias, out_dtype, y, x8_out, sx_out);
  GroupStrides s = {};
  s.b = N * K;
  s.sb = (int32_t)N;
  s.bias = (int32_t)N;
  finish_grouped_args(g, s);
  const Groups gr = {offsets, E, (int32_t)T};
  if (T > 0 && N > 0 && rows_fast_ok<kKContig>(g, s) && fuse_rows(g, x, T, E)) {
    by_input(x.dtype, [&](auto in) {
      launch_fused<decltype(in)::value>(g, FusedX{x.data, x8_out, sx_out}, &gr, s, stream);
    });
    return hip_status();
  }
  if (is_hp(x.dtype)) enqueue_rows(x.data, x.dtype, T, K, x8_out, sx_out, offsets + E, stream);
  if (T > 0 && N > 0)
    launch_rows<kKContig, kI8, kI8>(g, gr, s, GroupedSide{}, rows_tile<kKContig>(g, gr, s), stream);
  return hip_status();
}

}  // extern "C"
