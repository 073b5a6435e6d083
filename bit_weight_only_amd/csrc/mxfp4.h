// Element types and E8M0 / E2M1 values shared by the MXFP4 kernels and the
// expert dispatch.
#pragma once

#include "device.h"

namespace lbq {
namespace mxfp4 {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// lbq_dtype of include/lbq.h
constexpr int kF16 = 0, kBF16 = 1, kF32 = 2;

template <int DT>
struct Elem;
template <>
struct Elem<kF16> {
  using type = uint16_t;
};
template <>
struct Elem<kBF16> {
  using type = uint16_t;
};
template <>
struct Elem<kF32> {
  using type = float;
};

template <int DT>
__device__ __forceinline__ float to_f32(typename Elem<DT>::type v) {
  if constexpr (DT == kF16) return f16_bits_to_f32(v);
  else if constexpr (DT == kBF16) return __uint_as_float(static_cast<uint32_t>(v) << 16);
  else return v;
}
// one rounding, to nearest even
template <int DT>
__device__ __forceinline__ typename Elem<DT>::type from_f32(float v) {
  if constexpr (DT == kF16) return f32_to_f16_bits(v);
  else if constexpr (DT == kBF16) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  else return v;
}

// Eight consecutive values at unit (index / 8) of a 16-byte-aligned buffer.
template <int DT>
__device__ __forceinline__ void store8(void *out, size_t unit, const float v[8]) {
  if constexpr (DT == kF32) {
    float4_t *o = static_cast<float4_t *>(out) + 2 * unit;
    o[0] = float4_t{v[0], v[1], v[2], v[3]};
    o[1] = float4_t{v[4], v[5], v[6], v[7]};
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = from_f32<DT>(v[2 * i]) | (static_cast<uint32_t>(from_f32<DT>(v[2 * i + 1])) << 16);
    static_cast<uint4 *>(out)[unit] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// 2^(byte - 127) for byte <= 254 (byte 0: the subnormal 2^-127).
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}

// The value of one e2m1 code: magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6, sign in bit 3.
__device__ __forceinline__ float e2m1_value(uint32_t c) {
  // exponent and mantissa dropped into fp32's fields make the value times
  // 2^-126 (the subnormal case included); the product is exact
  const uint32_t bits = ((c & 8u) << 28) | ((c & 7u) << 22);
  return __uint_as_float(bits) * 0x1p+126f;
}

}  // namespace mxfp4
}  // namespace lbq
