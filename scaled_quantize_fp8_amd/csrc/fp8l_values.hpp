// Values of the high-precision types (kIn*): stores of fp32 values, rounded to
// nearest even (the counterparts of load1 and load8), and raw pieces.
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

// 16 bytes at any address that suits the type: gfx950 takes such wide accesses.
typedef uint32_t Any4 __attribute__((ext_vector_type(4), aligned(2)));

// 8 consecutive elements at any address that suits the type.
template <int IN>
FP8L_DEV void store8(void* p, int64_t i, const float v[8]) {
  Any4* const q = reinterpret_cast<Any4*>(reinterpret_cast<uint8_t*>(p) + i * (IN == kInF32 ? 4 : 2));
  if constexpr (IN == kInF32) {
    q[0] = Any4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                __float_as_uint(v[3])};
    q[1] = Any4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                __float_as_uint(v[7])};
  } else {
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = IN == kInF16 ? f32_to_f16(v[2 * j]) | (f32_to_f16(v[2 * j + 1]) << 16)
                          : pk_bf16(v[2 * j], v[2 * j + 1]);
    q[0] = Any4{o[0], o[1], o[2], o[3]};
  }
}

// N values (1, or 8 at any address that suits the type) as loaded, and in 32
// bits: several are in flight when all are loaded before the first is looked
// at.  ONCE: a streaming load (values that are read once).
template <int IN, int N>
struct Raw {
  static constexpr int kWords = N == 1 ? 1 : (IN == kInF32 ? 8 : 4);
  uint32_t w[kWords];
  FP8L_DEV void put(int j, float f) {  // of a value that the type holds
    if constexpr (N == 1 || IN == kInF32) w[j] = __float_as_uint(f);
    else {
      const uint32_t h = IN == kInBF16 ? __float_as_uint(f) >> 16 : f32_to_f16(f);
      w[j / 2] = j & 1 ? (w[j / 2] & 0xffffu) | (h << 16) : (w[j / 2] & 0xffff0000u) | h;
    }
  }
  template <bool ONCE = false>
  FP8L_DEV void load(const void* p, int64_t i) {
    if constexpr (N == 1) {
      w[0] = __float_as_uint(load1<IN>(p, i));
    } else {
      const Any4* const q = reinterpret_cast<const Any4*>(reinterpret_cast<const uint8_t*>(p) +
                                                          i * (IN == kInF32 ? 4 : 2));
#pragma unroll
      for (int j = 0; j < kWords / 4; ++j) {
        const Any4 x = ONCE ? __builtin_nontemporal_load(q + j) : q[j];
        w[4 * j] = x.x, w[4 * j + 1] = x.y, w[4 * j + 2] = x.z, w[4 * j + 3] = x.w;
      }
    }
  }
  FP8L_DEV void zero() {
#pragma unroll
    for (int j = 0; j < kWords; ++j) w[j] = 0;
  }
  FP8L_DEV float get(int j) const {
    if constexpr (N == 1 || IN == kInF32) return __uint_as_float(w[j]);
    else if constexpr (IN == kInBF16)
      return __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
    else return f16_to_f32((w[j / 2] >> (16 * (j & 1))) & 0xffffu);
  }
};

}  // namespace fp8l
