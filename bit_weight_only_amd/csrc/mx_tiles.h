// What the MXFP4 product kernels share: the row tiles of an expert-sorted list,
// operands of the matrix instruction, and stores.
#pragma once

#include "device.h"
#include "mxfp4.h"

namespace lbq {
namespace mxfp4 {

typedef int v8i_t __attribute__((ext_vector_type(8)));

// Row tiles of bm rows of an expert-sorted list; every expert may end in a
// ragged one. Each wave counts for itself: lane l holds the ranges of experts
// l per .. (l + 1) per - 1 (all loads at once) and the running sum of their
// tiles. offsets is taken as it comes: ranges are clamped to [0, T].
struct GroupTile {
  int e, i0, n;   // expert, first list row, rows
};
struct GroupTiles {
  static constexpr int kMost = 16;   // experts per lane, for up to 1024
  int at[kMost + 1];                 // where the lane's experts begin, and the last ends
  int per, bm, mine, incl;
  __device__ __forceinline__ GroupTiles(const int32_t *offsets, int E, int T, int bm_) : per((E + 63) / 64), bm(bm_) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i <= kMost; ++i)
      if (i <= per) at[i] = offsets[min(lane * per + i, E)];
    mine = 0;
#pragma unroll
    for (int i = 0; i <= kMost; ++i)
      if (i <= per) {
        at[i] = min(max(at[i], i > 0 ? at[i - 1] : 0), T);
        if (i > 0) mine += (at[i] - at[i - 1] + bm - 1) / bm;
      }
    incl = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int o = __shfl_up(incl, d);
      if (lane >= d) incl += o;
    }
  }
  __device__ __forceinline__ int total() const { return __builtin_amdgcn_readlane(incl, 63); }
  // tile number slot < total(), the same for every lane
  __device__ __forceinline__ GroupTile find(int slot) const {
    const int src = __builtin_ctzll(__ballot(slot < incl));
    int k = slot - (incl - mine), e = 0, i0 = 0, n = 0;   // of use in lane src
#pragma unroll
    for (int i = 0; i < kMost; ++i)
      if (i < per) {
        const int rows = at[i + 1] - at[i], tiles = (rows + bm - 1) / bm;
        if (k >= 0 && k < tiles) {
          e = src * per + i;
          i0 = at[i] + k * bm;
          n = min(rows - k * bm, bm);
        }
        k -= tiles;
      }
    return GroupTile{__builtin_amdgcn_readlane(e, src), __builtin_amdgcn_readlane(i0, src),
                     __builtin_amdgcn_readlane(n, src)};
  }
};

// Workgroups go to the eight XCDs in turn, each with an L2 of its own: XCD i
// takes the i-th eighth of `total` pieces of work in order, so that neighbours
// share an L2. The piece of workgroup pid, -1 for none.
__device__ __forceinline__ int xcd_order(int pid, int total) {
  const int xcd = pid & 7, at = pid >> 3, q = total / 8, rem = total % 8;
  return at < q + (xcd < rem ? 1 : 0) ? xcd * q + min(xcd, rem) + at : -1;
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
