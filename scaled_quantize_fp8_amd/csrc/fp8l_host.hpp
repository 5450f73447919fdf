// Host-side helpers shared by the library's translation units: argument
// checks, per-device caches, and the pieces of the quantize that other entry
// points than its own enqueue.
#pragma once

#include <limits.h>
#include <stdint.h>
#include <stdlib.h>

#include <atomic>

#include "../../include/fp8linear.h"
#include "fp8l_device.hpp"
#include "fp8l_gemm.hpp"
#include "fp8l_quantize.hpp"

namespace fp8l {

// Per-device host caches are atomics: library calls may come from several
// host threads, and two first calls on one device may both fill an entry
// (with the same value).
inline int cu_count() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
      n = 256;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Raise a kernel's dynamic LDS limit to lds bytes, once per device (the
// flag is published after the attribute is set, so a thread that sees it
// launches after the setting).
inline void set_lds_limit(const void* kernel, int lds, std::atomic<bool> (&done)[64]) {
  int dev = 0;
  const bool known = hipGetDevice(&dev) == hipSuccess && dev >= 0 && dev < 64;
  if (known && done[dev].load(std::memory_order_acquire)) return;
  (void)hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (known) done[dev].store(true, std::memory_order_release);
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline bool is_hp(int32_t dt) { return dt == FP8_DT_F32 || dt == FP8_DT_F16 || dt == FP8_DT_BF16; }
inline bool is_f8(int32_t dt) { return dt == FP8_DT_E4M3 || dt == FP8_DT_E5M2; }
inline bool valid_fmt(int32_t f) { return f == FP8_E4M3 || f == FP8_E5M2; }
inline int32_t fmt_dtype(int32_t f) { return f == FP8_E4M3 ? FP8_DT_E4M3 : FP8_DT_E5M2; }
inline int dtype_fmt(int32_t dt) { return dt == FP8_DT_E4M3 ? kE4M3 : kE5M2; }

// a * b fits in int64 (a, b >= 0)
inline bool mul_ok(int64_t a, int64_t b) { return a == 0 || b <= INT64_MAX / 4 / a; }

inline int check_ring(const fp8_ring_t* r) {
  if (!r) return FP8_OK;
  if (!r->dev) return FP8_ERR_NULL;
  if (r->hist_len < 1 || r->hist_len > FP8_RING_MAX_HIST) return FP8_ERR_RING;
  if (((uintptr_t)r->dev & 255u) != 0) return FP8_ERR_RING;
  return FP8_OK;
}

// a scale output must not be the ring's own scale slot
inline int check_alias(const fp8_ring_t* r, const float* scale_out) {
  if (r && scale_out && (const void*)scale_out >= r->dev &&
      (const char*)scale_out < (const char*)r->dev + sizeof(RingHdr))
    return FP8_ERR_RING;
  return FP8_OK;
}

// True while the stream is being captured into a graph.  A query that fails
// counts as not capturing (a launch on such a stream fails on its own).
inline bool capturing(hipStream_t st) {
  hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
  return hipStreamIsCapturing(st, &cs) == hipSuccess && cs == hipStreamCaptureStatusActive;
}

// A ring's first use seeds it with an extra amax pass, decided on the host
// from ring->seeded.  Captured into a graph, that pass and the seeding
// conversion would run again on every replay (dynamic scaling, while the
// host flag says seeded), so an unseeded ring is refused under capture.
inline int check_seed_capture(const fp8_ring_t* r, hipStream_t st) {
  return (r && !r->seeded && capturing(st)) ? FP8_ERR_RING : FP8_OK;
}

// Checks for one quantize (shared by the four entry points).
inline int check_quant(const void* x, int32_t in_dtype, int64_t n, int32_t fmt, const uint8_t* q,
                const fp8_ring_t* ring, const float* scale_used, const float* amax_out,
                hipStream_t stream) {
  if (n < 0) return FP8_ERR_SHAPE;
  if (!is_hp(in_dtype) || !valid_fmt(fmt)) return FP8_ERR_DTYPE;
  if (n > 0 && (!x || !q)) return FP8_ERR_NULL;
  if (!scale_used) return FP8_ERR_NULL;
  if (!ring && !amax_out) return FP8_ERR_NULL;
  int st = check_ring(ring);
  if (st) return st;
  if ((st = check_alias(ring, scale_used))) return st;
  return check_seed_capture(ring, stream);
}

// 2-D shape of a quantize: the column-sum variant (ws != null) or the
// transposed/dual variant (tkernel: q and/or qt).
struct ColsumSpec {
  int64_t rows, cols;
  float* ws;
  uint8_t* qt = nullptr;
  bool tkernel = false;
};


// A quantize through this ring may leave its fold to the GEMM that consumes
// the codes: the ring is seeded (one converting launch, no seeding pass) and
// its window fits the one wave that folds it.
inline bool can_defer(const fp8_ring_t* r) { return r && r->seeded && r->hist_len <= 64; }

// The fold the consuming GEMM does for a deferred quantize through r.
inline RingFold fold_of(const fp8_ring_t* r, int32_t fmt, float* amax_out) {
  RingFold f = {};
  f.ring = reinterpret_cast<RingHdr*>(r->dev);
  f.hist = reinterpret_cast<float*>(reinterpret_cast<char*>(r->dev) + sizeof(RingHdr));
  f.hist_len = r->hist_len;
  f.fmt_max = fmt == FP8_E4M3 ? FmtTraits<kE4M3>::kMax : FmtTraits<kE5M2>::kMax;
  f.amax_out = amax_out;
  return f;
}

inline int hip_status() { return hipGetLastError() == hipSuccess ? FP8_OK : FP8_ERR_HIP; }

// Tile choices; from kTile128x256 on of the grouped and integer layers only.
enum { kTileAuto = 0, kTile256x256, kTile256x128, kTile128x128, kTileV1, kTile256x256w8, kTile128x128w8,
       kTile128x256,
       kTileSkinny16, kTileSkinny32, kTileSkinny48, kTileSkinny64,
       kTileSkinny16Any, kTileSkinny32Any, kTileSkinny64Any };
int forced_tile();

// Defined in fp8l_api.hip.
bool enqueue_quant(const void* x, int32_t in_dtype, int64_t n, int32_t fmt, uint8_t* q,
                   fp8_ring_t* ring, float* scale_used, float* amax_out, const ColsumSpec* cs,
                   hipStream_t st, bool may_defer = false, const RowLimit& limit = RowLimit{});
// The amax pass alone: of a quantize that seeds ring, or (ring null) of a
// dynamic one, whose amax lands in amax_out.
void enqueue_amax(const void* x, int32_t dt, int64_t n, const fp8_ring_t* ring, float* amax_out,
                  const RowLimit& limit, hipStream_t st);

}  // namespace fp8l
