// Stores of fp32 values in the high-precision types (kIn*), rounded to
// nearest even: the counterparts of load1 and load8.
#pragma once

#include "fp8l_gemm.hpp"
#include "fp8l_quantize.hpp"

namespace fp8l {

template <int IN>
FP8L_DEV void store1(void* p, int64_t i, float v) {
  if constexpr (IN == kInF32) reinterpret_cast<float*>(p)[i] = v;
  else if constexpr (IN == kInF16) reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)f32_to_f16(v);
  else reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)f32_to_bf16(v);
}

// 8 consecutive elements, aligned as for load8.
template <int IN>
FP8L_DEV void store8(void* p, int64_t i, const float v[8]) {
  if constexpr (IN == kInF32) {
    float4* const q = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = IN == kInF16 ? f32_to_f16(v[2 * j]) | (f32_to_f16(v[2 * j + 1]) << 16)
                          : pk_bf16(v[2 * j], v[2 * j + 1]);
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + i) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

}  // namespace fp8l
