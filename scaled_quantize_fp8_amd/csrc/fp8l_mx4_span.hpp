// Which bytes the 4-bit kernels may touch: plain arithmetic of sizes and
// offsets, the same for the kernels and for a test on the CPU.
#pragma once

#include <stdint.h>

namespace fp8l {

// An offset past every buffer descriptor of these kernels: a load from it
// gives zeros.
constexpr uint32_t kMxNowhere = 0x80000000u;

// Bytes of scale words that a tile's descriptor covers: `rows` rows of each of
// `steps` steps, whose words lie `step` words apart (rows <= step, steps step <
// 2^29).  None without a step (K = 0): then the sum is no more than 0, the last
// step's number being -1.  32 bits and a maximum: a 64-bit choice here held up
// the kernel's first loads (33 rows of 11008 -> 4096 0.25 us).
constexpr uint32_t mx_scale_span(int32_t steps, int32_t step, int32_t rows) {
  const int32_t words = (steps - 1) * step + rows;
  return 4u * (uint32_t)(words > 0 ? words : 0);
}

// The codes of values [128 s + 8 sl, + 8) in a row of K (four bytes, with the
// scale word of their step); past the last value the row's first ones, which
// are not stored then.
struct MxPiece {
  int64_t step, byte;
};
constexpr MxPiece mx_piece(int64_t s, int sl, int64_t K) {
  return 128 * s + 8 * sl < K ? MxPiece{s, 64 * s + 4 * sl} : MxPiece{0, 0};
}

}  // namespace fp8l
