// What the adapters' kernels share: 16-bit operands of the matrix instructions,
// values held as several 16-bit pieces, and the tiles of tokens that belong to
// one adapter.
#pragma once

#include "device.h"
#include "kernels.h"
#include "mxfp4.h"

namespace lbq {
namespace adapters {

using namespace mxfp4;

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// Eight 16-bit values, one lane's share of an operand.
struct Oct {
  uint32_t w[4];
};
// The same in memory at any element (rows of N or r values start anywhere; the
// hardware takes 16-byte accesses at 2-byte addresses).
struct __attribute__((packed, aligned(2))) OctAnywhere {
  uint32_t w[4];
};

__device__ __forceinline__ Oct load_oct(const uint16_t *p) {
  const OctAnywhere v = *reinterpret_cast<const OctAnywhere *>(p);
  return {v.w[0], v.w[1], v.w[2], v.w[3]};
}
__device__ __forceinline__ Oct load_oct_aligned(const uint16_t *p) {
  const uint4 v = *reinterpret_cast<const uint4 *>(p);
  return {v.x, v.y, v.z, v.w};
}
__device__ __forceinline__ void store_oct(uint16_t *p, const Oct &v) {
  *reinterpret_cast<OctAnywhere *>(p) = {{v.w[0], v.w[1], v.w[2], v.w[3]}};
}
// the first `valid` of eight values, the rest zero; room: values to the buffer's end
__device__ __forceinline__ Oct load_oct_part(const uint16_t *p, int valid, size_t room) {
  Oct o{{0, 0, 0, 0}};
  if (valid <= 0) return o;
  if (room >= 8) {
    o = load_oct(p);
#pragma unroll
    for (int d = 0; d < 4; ++d) o.w[d] &= valid >= 2 * d + 2 ? ~0u : valid == 2 * d + 1 ? 0xFFFFu : 0u;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) o.w[i / 2] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
  }
  return o;
}

// D [16][16] += A [16][32] B [32][16]. Lane l gives row (column) l % 16 at k = 8 (l / 16)
// .. + 7 and holds D's column l % 16, rows 4 (l / 16) .. + 3.
template <int DT>
__device__ __forceinline__ float4_t mfma(const Oct &a, const Oct &b, float4_t c) {
  if constexpr (DT == kF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return from_f32<DT>(a) | static_cast<uint32_t>(from_f32<DT>(b)) << 16;
}

// PIECES 16-bit values whose sum is v[i] to 11 or 8 bits each (f16, bf16): out[p] holds
// the p-th pieces of the eight values. An fp32 sum enters a second product so, and
// loses no more than the second sum's own roundings (two pieces: 2^-21 and 2^-16 of
// it, below the result's own 2^-11 and 2^-8; three pieces of bf16: 2^-23).
template <int DT, int PIECES>
__device__ __forceinline__ void split8(const float v[8], Oct out[PIECES]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = v[2 * i], b = v[2 * i + 1];
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
      const uint32_t w = pack2<DT>(a, b);
      out[p].w[i] = w;
      if (p + 1 < PIECES) {
        a -= to_f32<DT>(static_cast<uint16_t>(w));
        b -= to_f32<DT>(static_cast<uint16_t>(w >> 16));
      }
    }
  }
}

// A power of two that brings magnitudes up to m into fp16's range with all of its
// bits to spare (m 2^e below 2^15), and its inverse; 1 for bf16, whose range is
// fp32's.
struct Scale {
  float to, back;
};
template <int DT>
__device__ __forceinline__ Scale scale_for(float m) {
  if constexpr (DT == kBF16) return {1.f, 1.f};
  const int ex = static_cast<int>(__float_as_uint(m) >> 23 & 255) - 127;
  const int e = min(max(14 - ex, -126), 126);
  return {__uint_as_float(static_cast<uint32_t>(127 + e) << 23), __uint_as_float(static_cast<uint32_t>(127 - e) << 23)};
}

// Tile number b of `rows` list entries each, adapter after adapter: its adapter
// (-1: past the last), first entry and count. One wavefront's lanes share the
// adapters; every lane gets the answer. Bad offsets give entries in [0, M) all
// the same.
struct Tile {
  int a, i0, n;
};
__device__ __forceinline__ Tile tile_of(const int32_t *__restrict__ offsets, int L, int M, int rows, int b) {
  const int lane = threadIdx.x & 63;
  const int per = (L + 63) / 64;
  const int first = min(lane * per, L), last = min(first + per, L);
  int tiles = 0;
  for (int a = first; a < last; ++a) {
    const int lo = min(max(offsets[a], 0), M), hi = min(max(offsets[a + 1], lo), M);
    tiles += (hi - lo + rows - 1) / rows;
  }
  int incl = tiles;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(incl, d);
    if (lane >= d) incl += o;
  }
  const uint64_t past = __ballot(incl > b);
  if (past == 0) return {-1, 0, 0};
  const int owner = __builtin_ctzll(past);
  Tile t{-1, 0, 0};
  if (lane == owner) {
    int at = incl - tiles;
    for (int a = first; a < last; ++a) {
      const int lo = min(max(offsets[a], 0), M), hi = min(max(offsets[a + 1], lo), M);
      const int n = (hi - lo + rows - 1) / rows;
      if (b < at + n) {
        t = {a, lo + (b - at) * rows, min(hi - lo - (b - at) * rows, rows)};
        break;
      }
      at += n;
    }
  }
  return {__builtin_amdgcn_readlane(t.a, owner), __builtin_amdgcn_readlane(t.i0, owner),
          __builtin_amdgcn_readlane(t.n, owner)};
}

}  // namespace adapters
}  // namespace lbq
