// Row-wise 8-bit integer quantize (one scale per token, or per output
// channel of a weight matrix):
//
//   s[r] = fl32(127 / max_k |x[r, k]|),   q[r, k] = rint(fl32(x[r, k] s[r])),
//
// rounding to the nearest integer, ties to even.  |x s| <= 127 (1 + 2^-23),
// so the codes need no clamp and -128 never appears.  s is the quantization
// multiplier, as in the FP8 quantize: the GEMMs multiply by 1 / s.
//   * a row of zeros, or one so small that 127 / max overflows: s = 1, codes 0;
//   * a row that holds a NaN or an infinity: s = NaN, codes 0, so that its
//     own outputs are NaN and no other row changes.
#pragma once

#include "fp8l_quantize.hpp"

namespace fp8l {

struct RowsArgs {
  const void* x;
  int8_t* q;
  float* scale;
  int64_t rows, cols;
  int32_t vec_ok;         // 16-byte loads and 8-byte stores of whole pieces
  const int32_t* valid;   // device row count, or null: all rows
};

FP8L_DEV float row_scale(uint32_t amax_bits) {
  if (amax_bits > 0x7f7fffffu) return __uint_as_float(0x7fc00000u);
  if (amax_bits == 0) return 1.0f;
  const float s = 127.0f / __uint_as_float(amax_bits);
  return s <= 3.402823466e38f ? s : 1.0f;
}

// Four values times s (ok: the row is finite) to four packed codes.
FP8L_DEV uint32_t i8x4(const float v[4], float s, bool ok) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w |= ((uint32_t)(int)__builtin_rintf(v[i] * s) & 0xffu) << (8 * i);
  return ok ? w : 0u;
}

// One block of NT threads per row, the row read twice (the second time from
// cache): 1024 threads where rows are few and long (33 rows of 11008: 4.7 us
// against 5.1 with 256), 256 where many rows share the CUs (4096 x 4096 bf16:
// 12.6 us, 4.0 TB/s).
template <int IN, int NT>
__global__ __launch_bounds__(NT) void quantize_rows_kernel(RowsArgs a) {
  __shared__ uint32_t sh[NT / 64];
  const int64_t rows = a.valid ? min<int64_t>(max(*a.valid, 0), a.rows) : a.rows;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const int64_t e0 = r * a.cols;
    uint32_t mx = 0;
    const int64_t nv = a.vec_ok ? a.cols / 8 : 0;
    for (int64_t c = threadIdx.x; c < nv; c += NT) {
      float v[8];
      load8<IN>(a.x, e0 + 8 * c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) mx = max(mx, absbits(v[i]));
    }
    for (int64_t c = 8 * nv + threadIdx.x; c < a.cols; c += NT)
      mx = max(mx, absbits(load1<IN>(a.x, e0 + c)));
    mx = block_max_u32<NT>(mx, sh);
    const float s = row_scale(mx);
    const bool ok = mx <= 0x7f7fffffu;
    if (threadIdx.x == 0) a.scale[r] = s;
    for (int64_t c = threadIdx.x; c < nv; c += NT) {
      float v[8];
      load8<IN>(a.x, e0 + 8 * c, v);
      *reinterpret_cast<uint2*>(a.q + e0 + 8 * c) = make_uint2(i8x4(v, s, ok), i8x4(v + 4, s, ok));
    }
    for (int64_t c = 8 * nv + threadIdx.x; c < a.cols; c += NT) {
      const float v[4] = {load1<IN>(a.x, e0 + c), 0.0f, 0.0f, 0.0f};
      a.q[e0 + c] = (int8_t)(i8x4(v, s, ok) & 0xffu);
    }
  }
}

}  // namespace fp8l
