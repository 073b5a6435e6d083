// What the MXFP4 product kernels share: the row tiles of an expert-sorted list,
// operands of the matrix instruction, and stores.
#pragma once

#include "device.h"
#include "mxfp4.h"

namespace lbq {
namespace mxfp4 {

typedef int v8i_t __attribute__((ext_vector_type(8)));

// Row tile `slot` of the expert-sorted list: its expert, first row and rows
// (0 rows past the last tile). Every lane of the wave gets the same answer.
// offsets is taken as it comes: ranges are clamped to [0, T].
struct GroupTile {
  int e, i0, n;
};
__device__ __forceinline__ GroupTile find_tile(const int32_t *offsets, int E, int T, int bm, int slot) {
  const int lane = threadIdx.x & 63;
  const int per = (E + 63) / 64, e0 = lane * per;
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int e = e0 + i;
    if (e >= E) break;
    const int lo = min(max(offsets[e], 0), T), hi = min(max(offsets[e + 1], lo), T);
    mine += (hi - lo + bm - 1) / bm;
  }
  int incl = mine;
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(incl, d);
    if (lane >= d) incl += o;
  }
  const uint64_t past = __ballot(slot < incl);
  GroupTile t{0, 0, 0};
  if (past == 0) return t;
  const int src = __builtin_ctzll(past);
  int k = slot - (incl - mine);   // the lane's own tile number, if src
  if (lane == src) {
    for (int i = 0; i < per; ++i) {
      const int e = e0 + i;
      if (e >= E) break;
      const int lo = min(max(offsets[e], 0), T), hi = min(max(offsets[e + 1], lo), T);
      const int tiles = (hi - lo + bm - 1) / bm;
      if (k < tiles) {
        t = GroupTile{e, lo + k * bm, min(hi - lo - k * bm, bm)};
        break;
      }
      k -= tiles;
    }
  }
  t.e = __shfl(t.e, src);
  t.i0 = __shfl(t.i0, src);
  t.n = __shfl(t.n, src);
  return t;
}

__device__ __forceinline__ v8i_t operand(uint4 v) {
  return v8i_t{static_cast<int>(v.x), static_cast<int>(v.y), static_cast<int>(v.z), static_cast<int>(v.w), 0, 0, 0, 0};
}

// Four neighbouring outputs n .. n + 3 of the row at element `row` of y.
__device__ __forceinline__ void store4(void *y, int dtype, size_t row, int n, int N, const float4_t &v) {
  if (dtype == kF32) {
    float *o = static_cast<float *>(y) + row + n;
    if (N % 4 == 0) {
      if (n < N) *reinterpret_cast<float4_t *>(o) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < N) o[i] = v[i];
    }
    return;
  }
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = dtype == kF16 ? from_f32<kF16>(v[i]) : from_f32<kBF16>(v[i]);
  uint16_t *o = static_cast<uint16_t *>(y) + row + n;
  if (N % 4 == 0) {
    if (n < N)
      *reinterpret_cast<uint2 *>(o) =
          make_uint2(h[0] | (static_cast<uint32_t>(h[1]) << 16), h[2] | (static_cast<uint32_t>(h[3]) << 16));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) o[i] = h[i];
  }
}

}  // namespace mxfp4
}  // namespace lbq
