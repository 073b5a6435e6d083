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

// The scale byte of a block whose largest magnitude has the bit pattern m (sign
// off; patterns of one type order like their magnitudes, infinities and NaN
// last). bf16 and fp32 values below the normal range have exponent field 0 and
// get byte 0, like every block whose exponent clamps at -127.
template <int DT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t m) {
  int e;   // fp32's exponent field of the magnitude
  bool finite;
  if constexpr (DT == kF16) {
    finite = m < 0x7C00u;
    e = static_cast<int>(__float_as_uint(f16_bits_to_f32(m)) >> 23);
  } else if constexpr (DT == kBF16) {
    finite = m < 0x7F80u;
    e = static_cast<int>(m >> 7);
  } else {
    finite = m < 0x7F800000u;
    e = static_cast<int>(m >> 23);
  }
  return finite ? static_cast<uint32_t>(max(e - 2, 0)) : 255u;
}

// Codes of eight values divided by the power of two s: 16-bit pairs in four
// words, or fp32. The conversion instruction divides, rounds once to nearest
// even and saturates.
template <int DT>
__device__ __forceinline__ uint32_t codes8(const uint32_t w[4], float s) {
  uint32_t o = 0;
  if constexpr (DT == kF16) {
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(o, __builtin_bit_cast(half2_t, w[0]), s, 0);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(o, __builtin_bit_cast(half2_t, w[1]), s, 1);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(o, __builtin_bit_cast(half2_t, w[2]), s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(o, __builtin_bit_cast(half2_t, w[3]), s, 3);
  } else {
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2_t, w[0]), s, 0);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2_t, w[1]), s, 1);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2_t, w[2]), s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2_t, w[3]), s, 3);
  }
}
__device__ __forceinline__ uint32_t codes8_f32(const float v[8], float s) {
  uint32_t o = 0;
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[0], v[1], s, 0);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[2], v[3], s, 1);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[4], v[5], s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[6], v[7], s, 3);
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
