// C entry points of the routing to experts and of the exchange of rows with
// them.  Checks run before the first launch; nothing is allocated.
#include "fp8l_host.hpp"
#include "fp8l_route.hpp"

namespace fp8l {
namespace {

// Slots of one chunk of the counting sort: 2048, or as many more as keep it at
// a chunk for each CU.  Every block adds up all chunks' counts, which limits
// their number: 2^20 slots in 256 experts 18 us, with up to 512 chunks 31, with
// 128 22.
constexpr int kMaxChunks = 256;
int plan_chunk(int64_t slots) {
  int64_t c = (slots + kMaxChunks - 1) / kMaxChunks;
  c = (c + kPlaceThreads - 1) / kPlaceThreads * kPlaceThreads;
  return (int)(c < 2048 ? 2048 : c);
}
int64_t plan_chunks(int64_t slots) {
  const int64_t c = plan_chunk(slots);
  return slots == 0 ? 1 : (slots + c - 1) / c;
}

// Slots that every block counts itself rather than wait for another launch:
// 32768 in 96 experts 6.6 us, one more, in two launches, 8.1.
constexpr int64_t kSelfSlots = 32768;
constexpr int kSelfChunk = kPlaceThreads;

// Slot numbers, and those of a last chunk's lanes behind them, stay below 2^31.
constexpr int64_t kMaxSlots = 1 << 30;

int check_slots(int64_t T, int64_t k) {
  if (T < 0 || k < 1 || k > kRouteMaxK || T > kMaxSlots / k) return FP8_ERR_SHAPE;
  return FP8_OK;
}
int check_route(int64_t T, int64_t E, int64_t k) {
  const int st = check_slots(T, k);
  if (st) return st;
  return E < 1 || E > kRouteMaxE || k > E ? FP8_ERR_SHAPE : FP8_OK;
}

template <class F>
void by_type(int32_t dt, F&& f) {
  if (dt == FP8_DT_F32) f(std::integral_constant<int, kInF32>{});
  else if (dt == FP8_DT_F16) f(std::integral_constant<int, kInF16>{});
  else f(std::integral_constant<int, kInBF16>{});
}

template <int N>
using Int = std::integral_constant<int, N>;

// Lanes per row and experts per lane: 16 lanes put four rows into a wave; 64
// are for more than 256 experts or 16 slots.
template <class F>
void by_row(int E, int k, F&& f) {
  if (E <= 256 && k <= 16) {
    if (E <= 16) f(Int<16>{}, Int<1>{});
    else if (E <= 64) f(Int<16>{}, Int<4>{});
    else if (E <= 128) f(Int<16>{}, Int<8>{});
    else f(Int<16>{}, Int<16>{});
  } else {
    if (E <= 256) f(Int<64>{}, Int<4>{});
    else if (E <= 512) f(Int<64>{}, Int<8>{});
    else f(Int<64>{}, Int<16>{});
  }
}

// Rows of one launch of the choice or of its gradient, up to 64 lanes each: a
// grid of 2^32 threads or more would wrap.  More rows take further launches;
// these start at multiples of 16 bytes where the first one does.
constexpr int64_t kPartRows = 1 << 24;
template <class F>
void by_parts(int64_t T, F&& f) {  // f(first row, rows)
  for (int64_t t = 0; t < T; t += kPartRows) f(t, T - t < kPartRows ? T - t : kPartRows);
}

void enqueue_plan(const int32_t* idx, int64_t T, int32_t k, int32_t E, int32_t* offsets,
                  int32_t* pos, void* ws, hipStream_t st) {
  const int64_t n = T * k;
  PlanArgs a = {idx, offsets, pos, reinterpret_cast<int32_t*>(ws), (int32_t)n, E,
                plan_chunk(n), (int32_t)plan_chunks(n)};
  if (n <= kSelfSlots) {
    a.counts = nullptr;
    a.chunk = kSelfChunk;
    a.chunks = n == 0 ? 1 : (int32_t)((n + kSelfChunk - 1) / kSelfChunk);
  }
  if (n > kSelfSlots)
    hipLaunchKernelGGL(plan_count_kernel, dim3(a.chunks), dim3(kRThreads), 0, st, a);
  hipLaunchKernelGGL(plan_place_kernel, dim3(a.chunks), dim3(kPlaceThreads),
                     place_lds<kPlaceThreads>(E), st, a);
}

int check_plan(int64_t T, int32_t k, int32_t E, const int32_t* offsets, const int32_t* pos,
               const void* ws) {
  if (!offsets || (T > 0 && !pos)) return FP8_ERR_NULL;
  const size_t need = fp8_route_workspace_bytes(T, E, k);
  if (need > 0 && !ws) return FP8_ERR_NULL;
  return ((uintptr_t)ws & 3u) != 0 ? FP8_ERR_SHAPE : FP8_OK;
}

// Pieces of a row over threads and blockIdx.y, tokens over blockIdx.x.
dim3 row_grid(int64_t T, int64_t pieces, RowGrid& g) {
  g.pieces = (int32_t)pieces;
  g.width_log = 0;
  while ((1 << g.width_log) < kRThreads && (1 << g.width_log) < pieces) ++g.width_log;
  const int64_t per = kRThreads >> g.width_log;
  const int64_t blocks = (T + per - 1) / per, cap = 1 << 20;
  return dim3((unsigned)(blocks < cap ? blocks : cap),
              (unsigned)((pieces + (1 << g.width_log) - 1) >> g.width_log));
}

// Rows of a buffer that slots point into, and of a row's values: blockIdx.y
// stays below 2^16 whatever the piece.
int check_rows(int64_t T, int32_t k, int64_t D, int64_t R) {
  const int st = check_slots(T, k);
  if (st) return st;
  if (D < 0 || D > (1 << 22) || R < 0 || R > INT32_MAX) return FP8_ERR_SHAPE;
  return FP8_OK;
}

}  // namespace
}  // namespace fp8l

using namespace fp8l;

extern "C" {

size_t fp8_route_workspace_bytes(int64_t T, int32_t E, int32_t k) {
  if (check_slots(T, k) || E < 1 || E > kRouteMaxE) return 0;
  return T * k > kSelfSlots ? (size_t)plan_chunks(T * k) * E * 4 : 0;
}

int fp8_route_fwd(int64_t T, int32_t E, int32_t k, const void* logits, int32_t dtype,
                  const float* bias, int32_t score, int32_t groups, int32_t groups_kept,
                  int32_t group_top, int32_t renorm, float scale, int32_t* idx, float* weights,
                  int32_t* offsets, int32_t* pos, void* ws, hipStream_t stream) {
  int st = check_route(T, E, k);
  if (st) return st;
  if (!is_hp(dtype) || (score != FP8_ROUTE_SOFTMAX && score != FP8_ROUTE_SIGMOID))
    return FP8_ERR_DTYPE;
  if (groups < 1 || E % groups != 0 || groups_kept < 1 || groups_kept > groups ||
      (group_top != 1 && group_top != 2) || groups_kept * (E / groups) < k)
    return FP8_ERR_SHAPE;
  if (T > 0 && (!logits || !idx || !weights)) return FP8_ERR_NULL;
  if ((offsets || pos) && (st = check_plan(T, k, E, offsets, pos, ws))) return st;
  RouteArgs a = {logits, bias, idx, weights, (int32_t)T, E, k, score == FP8_ROUTE_SIGMOID,
                 groups, groups_kept, group_top, renorm != 0, scale, 0, 0};
  bool placed = false;
  if (T > 0)
    by_type(dtype, [&](auto in) {
      by_row(E, k, [&](auto l, auto v) {
        constexpr int IN = decltype(in)::value, L = decltype(l)::value, V = decltype(v)::value;
        constexpr int per = kRThreads / L;
        const int size = dtype == FP8_DT_F32 ? 4 : 2, n = E / groups;
        a.vec = E % V == 0 && E * size % 16 == 0 && aligned16(logits) && aligned16(bias);
        // whole groups in 2^j lanes, or no limit by groups
        if (L == 16 && (groups == 1 || groups_kept == groups)) a.lanes = 16;
        else if (L == 16 && n % V == 0 && (n / V & (n / V - 1)) == 0) a.lanes = n / V;
        if constexpr (L == 16) {
          if (offsets && T <= kRoutePlaceRows) {
            const PlanArgs p = {idx, offsets, pos, nullptr, (int32_t)(T * k), E, kPlaceThreads, 1};
            static std::atomic<bool> lds_set[64];
            set_lds_limit((const void*)route_place_kernel<IN, V>, route_place_lds<V>(256),
                          lds_set);
            hipLaunchKernelGGL((route_place_kernel<IN, V>), dim3(1), dim3(kPlaceThreads),
                               route_place_lds<V>(E), stream, a, p);
            placed = true;
            return;
          }
        }
        by_parts(T, [&](int64_t t0, int64_t rows) {
          a.z = reinterpret_cast<const uint8_t*>(logits) + t0 * E * size;
          a.idx = idx + t0 * k;
          a.w = weights + t0 * k;
          a.T = (int32_t)rows;
          hipLaunchKernelGGL((route_kernel<IN, L, V>), dim3((unsigned)((rows + per - 1) / per)),
                             dim3(kRThreads), 0, stream, a);
        });
      });
    });
  if (offsets && !placed) enqueue_plan(idx, T, k, E, offsets, pos, ws, stream);
  return hip_status();
}

int fp8_route_bwd(int64_t T, int32_t E, int32_t k, const void* logits, int32_t dtype,
                  int32_t score, int32_t renorm, float scale, const int32_t* idx,
                  const float* dweights, void* dlogits, hipStream_t stream) {
  const int st = check_route(T, E, k);
  if (st) return st;
  if (!is_hp(dtype) || (score != FP8_ROUTE_SOFTMAX && score != FP8_ROUTE_SIGMOID))
    return FP8_ERR_DTYPE;
  if (T > 0 && (!logits || !idx || !dweights || !dlogits)) return FP8_ERR_NULL;
  if (T == 0) return FP8_OK;
  RouteBwdArgs a = {};
  a.r.E = E;
  a.r.k = k;
  a.r.score = score == FP8_ROUTE_SIGMOID;
  a.r.renorm = renorm != 0;
  a.r.scale = scale;
  by_type(dtype, [&](auto in) {
    by_row(E, k, [&](auto l, auto v) {
      constexpr int IN = decltype(in)::value, L = decltype(l)::value, V = decltype(v)::value;
      constexpr int per = kRThreads / L;
      by_parts(T, [&](int64_t t0, int64_t rows) {
        const int64_t at = t0 * E * (dtype == FP8_DT_F32 ? 4 : 2);
        a.r.z = reinterpret_cast<const uint8_t*>(logits) + at;
        a.r.idx = const_cast<int32_t*>(idx) + t0 * k;
        a.r.T = (int32_t)rows;
        a.dw = dweights + t0 * k;
        a.dz = reinterpret_cast<uint8_t*>(dlogits) + at;
        hipLaunchKernelGGL((route_bwd_kernel<IN, L, V>), dim3((unsigned)((rows + per - 1) / per)),
                           dim3(kRThreads), 0, stream, a);
      });
    });
  });
  return hip_status();
}

int fp8_route_plan(int64_t T, int32_t E, int32_t k, const int32_t* idx, int32_t* offsets,
                   int32_t* pos, void* ws, hipStream_t stream) {
  int st = check_slots(T, k);
  if (st) return st;
  if (E < 1 || E > kRouteMaxE) return FP8_ERR_SHAPE;
  if (T > 0 && !idx) return FP8_ERR_NULL;
  if ((st = check_plan(T, k, E, offsets, pos, ws))) return st;
  enqueue_plan(idx, T, k, E, offsets, pos, ws, stream);
  return hip_status();
}

int fp8_route_gather(int64_t T, int32_t k, int64_t row_bytes, int64_t R, const void* x,
                     const int32_t* pos, void* out, hipStream_t stream) {
  const int st = check_rows(T, k, 0, R);
  if (st) return st;
  if (row_bytes < 0 || row_bytes >= 1 << 24) return FP8_ERR_SHAPE;
  if (T == 0 || row_bytes == 0 || R == 0) return FP8_OK;
  if (!x || !pos || !out) return FP8_ERR_NULL;
  GatherArgs a = {reinterpret_cast<const uint8_t*>(x), reinterpret_cast<uint8_t*>(out), pos,
                  (int32_t)T, k, (int32_t)R, row_bytes, {}};
  auto go = [&](auto u) {
    constexpr int U = decltype(u)::value;
    const dim3 grid = row_grid(T, (row_bytes + U - 1) / U, a.grid);
    hipLaunchKernelGGL((gather_kernel<U>), grid, dim3(kRThreads), 0, stream, a);
  };
  if (row_bytes >= 16) go(Int<16>{});
  else go(Int<1>{});
  return hip_status();
}

int fp8_route_combine(int64_t T, int32_t k, int64_t D, int64_t R, const void* y, int32_t dtype,
                      const int32_t* pos, const float* weights, void* out, hipStream_t stream) {
  const int st = check_rows(T, k, D, R);
  if (st) return st;
  if (!is_hp(dtype)) return FP8_ERR_DTYPE;
  if (T == 0 || D == 0) return FP8_OK;
  if ((R > 0 && !y) || !pos || !out) return FP8_ERR_NULL;
  CombineArgs a = {y, pos, weights, out, (int32_t)T, k, (int32_t)R, D, {}};
  const bool vec = D >= 8;
  by_type(dtype, [&](auto in) {
    constexpr int IN = decltype(in)::value;
    const dim3 grid = row_grid(T, vec ? (D + 7) / 8 : D, a.grid);
    const bool uni = a.grid.width_log >= 6;  // a wave's pieces are one token's
    auto go = [&](auto n, auto u) {
      hipLaunchKernelGGL((combine_kernel<IN, decltype(n)::value, decltype(u)::value>), grid,
                         dim3(kRThreads), 0, stream, a);
    };
    if (vec && uni) go(Int<8>{}, std::true_type{});
    else if (vec) go(Int<8>{}, std::false_type{});
    else go(Int<1>{}, std::false_type{});
  });
  return hip_status();
}

int fp8_route_combine_bwd(int64_t T, int32_t k, int64_t D, int64_t R, const void* dout,
                          const void* y, int32_t dtype, const int32_t* pos, const float* weights,
                          void* dy, float* dweights, hipStream_t stream) {
  const int st = check_rows(T, k, D, R);
  if (st) return st;
  if (!is_hp(dtype)) return FP8_ERR_DTYPE;
  if (T == 0) return FP8_OK;
  if (!pos || !weights || (D > 0 && !dout) || (D > 0 && R > 0 && dweights && !y)) return FP8_ERR_NULL;
  CombineBwdArgs a = {dout, y, pos, weights, dy, dweights, (int32_t)T, k, (int32_t)R, D};
  const bool vec = D >= 8;
  const int64_t blocks = (T + 3) / 4, cap = 1 << 20;
  const dim3 grid((unsigned)(blocks < cap ? blocks : cap));
  by_type(dtype, [&](auto in) {
    constexpr int IN = decltype(in)::value;
    if (vec) hipLaunchKernelGGL((combine_bwd_kernel<IN, 8>), grid, dim3(kRThreads), 0, stream, a);
    else hipLaunchKernelGGL((combine_bwd_kernel<IN, 1>), grid, dim3(kRThreads), 0, stream, a);
  });
  return hip_status();
}

}  // extern "C"
