// C entry points of the linear layers in microscaled 4-bit floating point,
// dense and over ragged groups of rows.  Checks run before the first launch;
// nothing is allocated.
#include <type_traits>

#include "fp8l_grouped_host.hpp"
#include "fp8l_mx4_tile.hpp"

namespace fp8l {
namespace {

// 256 rows of codes stay below 2^31 bytes, a matrix' scale words below 2^29:
// the offsets inside a buffer resource.
constexpr int64_t kMxMaxK = (1 << 24) - 1;
constexpr int64_t kMxMaxWords = 1 << 29;

int64_t mx_blocks(int64_t K) { return (K + 31) / 32; }
int64_t mx_steps(int64_t K) { return (K + 127) / 128; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

int check_mx(int64_t rows, int64_t K) {
  if (rows < 0 || K < 0 || K > kMxMaxK || rows > INT32_MAX) return FP8_ERR_SHAPE;
  return mx_steps(K) > 0 && rows >= kMxMaxWords / mx_steps(K) ? FP8_ERR_SHAPE : FP8_OK;
}

template <class F>
void by_type(int32_t dt, F&& f) {
  if (dt == FP8_DT_F32) f(std::integral_constant<int, kInF32>{});
  else if (dt == FP8_DT_F16) f(std::integral_constant<int, kInF16>{});
  else f(std::integral_constant<int, kInBF16>{});
}

// Tiles of 16 rows (fewer where there are no more); along K, `unroll` steps at
// a time, as many blocks side by side as give the chip about 16 per CU.
dim3 quant_grid(int64_t mats, int64_t rows, int64_t steps, int unroll, int32_t* rows_log) {
  int log = 0;
  while (log < 4 && (1 << log) < rows) ++log;
  *rows_log = log;
  const int64_t bx = (rows + (1 << log) - 1) >> log, cap = 1 << 20;
  const int64_t across = (16 >> log) * unroll, most = (steps + across - 1) / across;
  int64_t by = (16 * cu_count() + bx * mats - 1) / (bx * mats);
  by = by < most ? by : most;
  return dim3((unsigned)(bx < cap ? bx : cap), (unsigned)(by < 65535 ? by : 65535), (unsigned)mats);
}

void enqueue_mx_quantize(const void* x, int32_t dt, int64_t mats, int64_t rows, int64_t K,
                         uint8_t* codes, uint8_t* scales, const int32_t* valid, hipStream_t st) {
  if (mats == 0 || rows == 0 || K == 0) return;
  MxQuantArgs a = {x, codes, reinterpret_cast<uint32_t*>(scales), rows, K, (int32_t)mx_steps(K),
                   (int32_t)mx_blocks(K), 0, valid};
  const bool vec = K % 8 == 0;
  const dim3 grid = quant_grid(mats, rows, a.steps, dt == FP8_DT_F32 ? 2 : 4, &a.rows_log);
  by_type(dt, [&](auto in) {
    constexpr int IN = decltype(in)::value;
    if (vec) hipLaunchKernelGGL((mx4_quantize_kernel<IN, true>), grid, dim3(kMxThreads), 0, st, a);
    else hipLaunchKernelGGL((mx4_quantize_kernel<IN, false>), grid, dim3(kMxThreads), 0, st, a);
  });
}

int check_linear(int64_t M, int64_t N, int64_t K, const void* x, int32_t x_dtype,
                 const uint8_t* x_scales, const uint8_t* w, const uint8_t* w_scales,
                 int32_t out_dtype, const void* y, const uint8_t* x4_out, const uint8_t* sx_out) {
  if (out_dtype != FP8_DT_BF16 && out_dtype != FP8_DT_F16) return FP8_ERR_DTYPE;
  if (!is_hp(x_dtype) && x_dtype != FP8_DT_MX4) return FP8_ERR_DTYPE;
  const bool hp = is_hp(x_dtype);
  const void* const xc = hp ? x4_out : x;
  const uint8_t* const xs = hp ? sx_out : x_scales;
  if (M > 0 && K > 0 && (!x || !xc || !xs)) return FP8_ERR_NULL;
  if (N > 0 && K > 0 && (!w || !w_scales)) return FP8_ERR_NULL;
  if (M > 0 && N > 0 && !y) return FP8_ERR_NULL;
  if (!aligned16(xc) || !aligned4(xs) || !aligned16(w) || !aligned4(w_scales)) return FP8_ERR_SHAPE;
  return FP8_OK;
}

MxArgs mx_args(int64_t M, int64_t N, int64_t K, const void* x, int32_t x_dtype,
               const uint8_t* x_scales, const uint8_t* w, const uint8_t* w_scales, const void* bias,
               int32_t out_dtype, void* y, const uint8_t* x4_out, const uint8_t* sx_out) {
  MxArgs g = {};
  g.a = is_hp(x_dtype) ? x4_out : reinterpret_cast<const uint8_t*>(x);
  g.sa = reinterpret_cast<const uint32_t*>(is_hp(x_dtype) ? sx_out : x_scales);
  g.b = w;
  g.sb = reinterpret_cast<const uint32_t*>(w_scales);
  g.ld = 16 * mx_blocks(K);
  g.sa_step = M;
  g.sb_step = N;
  g.M = M;
  g.N = N;
  g.steps = (int32_t)mx_steps(K);
  g.c = reinterpret_cast<uint16_t*>(y);
  g.ldc = N;
  g.bias = reinterpret_cast<const uint16_t*>(bias);
  g.out_f16 = out_dtype == FP8_DT_F16;
  g.c_vec = aligned16(y) && N % 8 == 0;
  return g;
}

template <int WGM>
void launch_tile(MxArgs& g, const Groups* gr, const MxStrides& s, hipStream_t st) {
  using T = MxTile<WGM>;
  static std::atomic<bool> set_dense[64], set_groups[64];
  g.tiles_n = (int32_t)((g.N + T::kBN - 1) / T::kBN);
  if (gr) {
    set_lds_limit((const void*)mx4_tile_groups_kernel<WGM>, T::kLds, set_groups);
    const int64_t most = (most_units(gr->T, gr->E, T::kBM) * g.tiles_n + 7) & ~7LL;
    hipLaunchKernelGGL((mx4_tile_groups_kernel<WGM>), dim3((unsigned)most), dim3(T::kThreads),
                       T::kLds, st, g, *gr, s);
  } else {
    set_lds_limit((const void*)mx4_tile_kernel<WGM>, T::kLds, set_dense);
    g.tiles_m = (int32_t)((g.M + T::kBM - 1) / T::kBM);
    hipLaunchKernelGGL((mx4_tile_kernel<WGM>), dim3((unsigned)g.tiles_m * (unsigned)g.tiles_n),
                       dim3(T::kThreads), T::kLds, st, g);
  }
}

// Waves that split K in a skinny launch of `waves` tile columns: doubled while
// the chip has room for more of them and each keeps two pieces (one row of
// 11008 -> 4096 22.6 us unsplit, 8.6 by four, 7.6 by eight; 32 rows of 4096 ->
// 32000, with 2000 tile columns, 13.6 unsplit, 14.8 by two); two of more than 8
// pieces where columns wait in line (16 experts of 4096 -> 11008, one row
// each: 53.2 unsplit, 49.5 by two, 50.9 by four).
int mx_split(int64_t waves, int64_t steps) {
  const int64_t pieces = (steps + 1) / 2;
  if (waves > 2048) return pieces > 8 ? 2 : 1;
  int kw = 1;
  while (kw < 8 && waves * kw <= 1536 && pieces >= 2 * kw) kw *= 2;
  return kw;
}

// Whether a kernel's blocks for T rows in E groups fit a launch.
bool mx_fits(int tile, int64_t T, int64_t E, int64_t N, int64_t K) {
  const int64_t n256 = (N + 255) / 256;
  if (tile == kTile128x256) return grid_fits(most_units(T, E, 128) * n256, 256);
  if (tile == kTile256x256w8) return grid_fits(most_units(T, E, 256) * n256, 512);
  const int mt = tile - kTileSkinny16 + 1;
  const int64_t units = most_units(T, E, 16 * mt), cols = (N + 15) / 16;
  const int jw = 8 / mx_split(units * cols, mx_steps(K));
  return grid_fits(units * ((cols + jw - 1) / jw), 512);
}

template <int MT>
void launch_skinny(MxArgs& g, const Groups* gr, const MxStrides& s, hipStream_t st) {
  const int64_t units = gr ? most_units(gr->T, gr->E, 16 * MT) : (g.M + 16 * MT - 1) / (16 * MT);
  const int64_t cols = (g.N + 15) / 16;
  const int kw = mx_split(units * cols, g.steps);
  const int lds = MxSkinny<MT>::kLds;
  g.tiles_n = (int32_t)((cols + 8 / kw - 1) / (8 / kw));
  if (gr)
    hipLaunchKernelGGL((mx4_skinny_groups_kernel<MT>),
                       dim3((unsigned)((units * g.tiles_n + 7) & ~7LL)), dim3(512), lds, st, g, *gr,
                       s, kw);
  else
    hipLaunchKernelGGL((mx4_skinny_kernel<MT>), dim3((unsigned)(units * g.tiles_n)), dim3(512), lds,
                       st, g, kw);
}

// Whether a call's blocks quantize its X themselves (MxFused).  Every block of
// 16 columns or more does all of it again, where the launch that it saves takes
// 2 to 3 us (bf16, us fused / in two launches: one row of 4096 -> 11008 6.6 /
// 10.1, of 11008 -> 4096 8.0 / 10.0; four rows of 1536 -> 6912 4.5 / 7.1, of 4096
// -> 11008 8.4 / 10.0, of 6912 -> 1536 7.5 / 8.0; eight of 4096 -> 11008 10.9 /
// 10.1).  The blocks do it side by side, so the bound is on a block's own work,
// rows K, whatever N is: one row of 4096 -> 128 3.9 / 7.0, of 4096 -> 32000 12.5 /
// 15.7, four of 1536 -> 100000 15.5 / 18.9; at the bound, seven of 4096 -> 512 7.0 /
// 7.3, of 4096 -> 32000 15.9 / 16.1, one of 28672 -> 4096 15.5 / 15.3.
// Groups: two rows per expert on average (any unit may have 16, whose
// codes must leave room for two blocks per CU; 24 rows, 64 experts of 1536 ->
// 6912 19.3 / 22.6; 16 rows, 16 of 4096 -> 11008 52.2 / 55.1).  groups 0: dense.
bool fuse_x(const void* x, int32_t dt, int64_t rows, int64_t groups, int64_t N, int64_t K) {
  if (!is_hp(dt) || K == 0 || K % 8 != 0 || !aligned16(x) || forced_tile() != kTileAuto) return false;
  if (!mx_fits(kTileSkinny16, rows, groups ? groups : 1, N, K)) return false;
  if (groups == 0) return rows <= 16 && rows * K <= 28672;
  return rows <= 2 * groups && K <= 4096;
}

template <int IN>
void launch_fused(MxArgs& g, const MxFusedX& fx, const Groups* gr, const MxStrides& s,
                  hipStream_t st) {
  const int64_t units = gr ? most_units(gr->T, gr->E, 16) : 1, cols = (g.N + 15) / 16;
  const int kw = mx_split(units * cols, g.steps);
  const int lds = MxFused<IN>::lds(gr ? 16 : (int)g.M, g.ld, g.steps);
  g.tiles_n = (int32_t)((cols + 8 / kw - 1) / (8 / kw));
  if (gr)
    hipLaunchKernelGGL((mx4_fused_groups_kernel<IN>),
                       dim3((unsigned)((units * g.tiles_n + 7) & ~7LL)), dim3(512), lds, st, g, fx,
                       *gr, s, kw);
  else
    hipLaunchKernelGGL((mx4_fused_kernel<IN>), dim3((unsigned)g.tiles_n), dim3(512), lds, st, g, fx,
                       kw);
}

// Microseconds of the kernels, from fits to a sweep of 8 to 8192 rows over six
// layer shapes, dense and in 8 and 64 groups; `steps` of 128 values of K.
//   skinny, 16 / 32 / 48 / 64 rows a unit: 4 + units N K (0.72 / 0.85 / 1.15 /
//     1.45) 1e-7: 32 rows of 4096 -> 11008 8.8 (7.8), 64 12.1 (10.5), 128 19.7
//     (17.1), 192 26.2 (23.6); 64 of 11008 -> 4096 10.3 (10.5); 64 rows in 64
//     groups of 1536 -> 6912 30.3 (34.7)
//   128x256, one block per CU: 5.5 + 0.635 steps: K = 1536 / 4096 / 11008 13.6 /
//     26.5 / 60 (13.1 / 25.8 / 60.1); two blocks per CU: a full round of 512
//     tiles takes 1.4 steps, fewer tiles at least 0.8 of it: 688 tiles of
//     K = 4096 67 (65), 1376 126 (125); not below the bytes of W at 5 TB/s
//   256x256: a full round 1.2 steps, a part of one 0.7 + 0.5 its share (under
//     the power limit busy CUs slow each other): 129 / 344 / 688 tiles of
//     K = 4096 34 / 69 / 121 (35 / 71 / 115)
// The fastest of those that fit a launch, 0: none does.
int mx_tile(int64_t rows, int64_t E, int64_t N, int64_t K) {
  const int f = forced_tile();
  if ((f == kTile256x256w8 || f == kTile128x256 || (f >= kTileSkinny16 && f <= kTileSkinny64)) &&
      mx_fits(f, rows, E, N, K))
    return f;
  const double cus = cu_count(), steps = (double)mx_steps(K), nk = (double)N * (double)K;
  const double per[4] = {0.72e-7, 0.85e-7, 1.15e-7, 1.45e-7};
  int best = 0;
  double us = 1e300;
  auto offer = [&](int tile, double t) {
    if (t < us && mx_fits(tile, rows, E, N, K)) us = t, best = tile;
  };
  for (int mt = 1; mt <= 4; ++mt)
    offer(kTileSkinny16 + mt - 1, 4 + expected_units(rows, E, 16 * mt) * nk * per[mt - 1]);
  const double n256 = (double)((N + 255) / 256), bytes = expected_units(rows, E, 1 << 30) * nk * 0.53;
  const double t128 = expected_units(rows, E, 128) * n256;
  double t = t128 <= cus ? 5.5 + 0.635 * steps
                         : 5 + (t128 < 1.6 * cus ? 0.8 : t128 / (2 * cus)) * 1.4 * steps;
  offer(kTile128x256, t < 4 + bytes / 5e6 ? 4 + bytes / 5e6 : t);
  const double rounds = expected_units(rows, E, 256) * n256 / cus, full = floor(rounds);
  t = 5 + (1.2 * full + (rounds > full ? 0.7 + 0.5 * (rounds - full) : 0)) * steps;
  offer(kTile256x256w8, t < 4 + bytes / 5e6 ? 4 + bytes / 5e6 : t);
  return best;
}

void launch_product(int tile, MxArgs& g, const Groups* gr, const MxStrides& s, hipStream_t st) {
  switch (tile) {
    case kTileSkinny16: return launch_skinny<1>(g, gr, s, st);
    case kTileSkinny32: return launch_skinny<2>(g, gr, s, st);
    case kTileSkinny48: return launch_skinny<3>(g, gr, s, st);
    case kTileSkinny64: return launch_skinny<4>(g, gr, s, st);
    case kTile128x256: return launch_tile<1>(g, gr, s, st);
    default: return launch_tile<2>(g, gr, s, st);
  }
}

}  // namespace
}  // namespace fp8l

using namespace fp8l;

extern "C" {

size_t fp8_mx4_code_bytes(int64_t rows, int64_t K) {
  return check_mx(rows, K) ? 0 : (size_t)(rows * mx_blocks(K) * 16);
}

size_t fp8_mx4_scale_bytes(int64_t rows, int64_t K) {
  return check_mx(rows, K) ? 0 : (size_t)(rows * mx_steps(K) * 4);
}

int fp8_mx4_quantize(const void* x, int32_t in_dtype, int64_t mats, int64_t rows, int64_t K,
                     uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  if (mats < 0 || mats > 65535) return FP8_ERR_SHAPE;
  const int st = check_mx(rows, K);
  if (st) return st;
  if (!is_hp(in_dtype)) return FP8_ERR_DTYPE;
  if (mats == 0 || rows == 0 || K == 0) return FP8_OK;
  if (!x || !codes || !scales) return FP8_ERR_NULL;
  if (!aligned16(codes) || !aligned4(scales)) return FP8_ERR_SHAPE;
  enqueue_mx_quantize(x, in_dtype, mats, rows, K, codes, scales, nullptr, stream);
  return hip_status();
}

int fp8_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t mats, int64_t rows,
                       int64_t K, void* out, int32_t out_dtype, hipStream_t stream) {
  if (mats < 0 || mats > 65535) return FP8_ERR_SHAPE;
  const int st = check_mx(rows, K);
  if (st) return st;
  if (!is_hp(out_dtype)) return FP8_ERR_DTYPE;
  if (mats == 0 || rows == 0 || K == 0) return FP8_OK;
  if (!codes || !scales || !out) return FP8_ERR_NULL;
  if (!aligned16(codes) || !aligned4(scales)) return FP8_ERR_SHAPE;
  MxDequantArgs a = {codes, reinterpret_cast<const uint32_t*>(scales), out, rows, K,
                     (int32_t)mx_steps(K), (int32_t)mx_blocks(K), 0, 0};
  a.vec = K % 8 == 0;
  const dim3 grid = quant_grid(mats, rows, a.steps, 4, &a.rows_log);
  by_type(out_dtype, [&](auto in) {
    hipLaunchKernelGGL((mx4_dequantize_kernel<decltype(in)::value>), grid, dim3(kMxThreads), 0,
                       stream, a);
  });
  return hip_status();
}

int fp8_mx4_linear_fwd(int64_t M, int64_t N, int64_t K, const void* x, int32_t x_dtype,
                       const uint8_t* x_scales, const uint8_t* w, const uint8_t* w_scales,
                       const void* bias, int32_t out_dtype, void* y, uint8_t* x4_out,
                       uint8_t* sx_out, hipStream_t stream) {
  int st = check_mx(M, K);
  if (st || (st = check_mx(N, K))) return st;
  if (!mul_ok(M, N)) return FP8_ERR_SHAPE;
  const int tile = M > 0 && N > 0 ? mx_tile(M, 1, N, K) : 1;
  if (tile == 0) return FP8_ERR_SHAPE;
  if ((st = check_linear(M, N, K, x, x_dtype, x_scales, w, w_scales, out_dtype, y, x4_out, sx_out)))
    return st;
  MxArgs g = mx_args(M, N, K, x, x_dtype, x_scales, w, w_scales, bias, out_dtype, y, x4_out, sx_out);
  if (M > 0 && N > 0 && fuse_x(x, x_dtype, M, 0, N, K)) {
    by_type(x_dtype, [&](auto in) {
      const MxFusedX fx = {x, K, x4_out, reinterpret_cast<uint32_t*>(sx_out)};
      launch_fused<decltype(in)::value>(g, fx, nullptr, MxStrides{}, stream);
    });
    return hip_status();
  }
  if (is_hp(x_dtype)) enqueue_mx_quantize(x, x_dtype, 1, M, K, x4_out, sx_out, nullptr, stream);
  if (M == 0 || N == 0) return hip_status();
  launch_product(tile, g, nullptr, MxStrides{}, stream);
  return hip_status();
}

int fp8_mx4_grouped_linear_fwd(int64_t T, int32_t E, int64_t N, int64_t K, const int32_t* offsets,
                               const void* x, int32_t x_dtype, const uint8_t* x_scales,
                               const uint8_t* w, const uint8_t* w_scales, const void* bias,
                               int32_t out_dtype, void* y, uint8_t* x4_out, uint8_t* sx_out,
                               hipStream_t stream) {
  int st = check_grouped(T, E, N, K);
  if (st || (st = check_mx(T, K)) || (st = check_mx(N, K))) return st;
  const int tile = T > 0 && N > 0 ? mx_tile(T, E, N, K) : 1;
  if (tile == 0) return FP8_ERR_SHAPE;
  if (!offsets) return FP8_ERR_NULL;
  if ((st = check_linear(T, N, K, x, x_dtype, x_scales, w, w_scales, out_dtype, y, x4_out, sx_out)))
    return st;
  MxArgs g = mx_args(T, N, K, x, x_dtype, x_scales, w, w_scales, bias, out_dtype, y, x4_out, sx_out);
  const MxStrides s = {N * g.ld, N * g.steps, N};
  const Groups gr = {offsets, E, (int32_t)T};
  if (T > 0 && N > 0 && fuse_x(x, x_dtype, T, E, N, K)) {
    by_type(x_dtype, [&](auto in) {
      const MxFusedX fx = {x, K, x4_out, reinterpret_cast<uint32_t*>(sx_out)};
      launch_fused<decltype(in)::value>(g, fx, &gr, s, stream);
    });
    return hip_status();
  }
  if (is_hp(x_dtype))
    enqueue_mx_quantize(x, x_dtype, 1, T, K, x4_out, sx_out, offsets + E, stream);
  if (T == 0 || N == 0) return hip_status();
  launch_product(tile, g, &gr, s, stream);
  return hip_status();
}

}  // extern "C"
