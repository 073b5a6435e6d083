// Low-rank adapters of many requests beside a shared projection. Token t with
// adapter a = ids[t], scale s_a:
//
//   h_t = x_t A_a^T        y_t = base_t + s_a h_t B_a^T
//
// in two launches; nothing uses atomics, so repeated calls give identical bits.
#include "adapters.h"

#include <algorithm>

namespace lbq {

namespace {

using namespace adapters;

constexpr int kThreads = 256, kWaves = kThreads / 64;

__device__ __forceinline__ int adapter_of(const int32_t *ids, int t, int L) {
  const int a = ids[t];
  return a >= 0 && a < L ? a : -1;
}

// ------------------------------------------------------------------ x A^T

// part[s][row][j] = sum over the s-th share of K of x[token(row)][k] A[a][j][k], a
// tile of up to 16 TF tokens of one adapter per workgroup column. BY_TOKEN: every
// token is a tile of its own, and a row its number; else rows are list entries.
//
// Both operands are contiguous along k, so they go from memory into the matrix
// instruction as they are. The waves take blocks of 128 values in turn, and add
// up at the end. Rows and columns past the last are copies of the last (their
// results are dropped), so nothing is masked.
template <int DT, int TF, int RF, bool BY_TOKEN>
__global__ void __launch_bounds__(kThreads) adapters_shrink_kernel(const uint16_t *__restrict__ x, int M, int K, int r,
                                                                   const uint16_t *__restrict__ A, int L,
                                                                   const int32_t *__restrict__ ids,
                                                                   const int32_t *__restrict__ offsets,
                                                                   const int32_t *__restrict__ perm,
                                                                   float *__restrict__ part) {
  __shared__ float4_t red[(kWaves - 1) * TF * RF * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
  Tile tile;
  if constexpr (BY_TOKEN) tile = {adapter_of(ids, blockIdx.x, L), static_cast<int>(blockIdx.x), 1};
  else tile = tile_of(offsets, L, M, 16 * TF, blockIdx.x);
  if (tile.a < 0) return;
  const uint16_t *xr[TF], *wr[RF];
#pragma unroll
  for (int f = 0; f < TF; ++f) {
    int t = tile.i0 + min(16 * f + col, tile.n - 1);
    if constexpr (!BY_TOKEN) t = min(max(perm[t], 0), M - 1);
    xr[f] = x + static_cast<size_t>(t) * K + 8 * q;
  }
#pragma unroll
  for (int f = 0; f < RF; ++f)
    wr[f] = A + (static_cast<size_t>(tile.a) * r + min(16 * f + col, r - 1)) * K + 8 * q;
  float4_t acc[TF][RF] = {};
  const int blocks = K / 128, splits = gridDim.y;
  const int lo = static_cast<int>(static_cast<long>(blocks) * blockIdx.y / splits);
  const int hi = static_cast<int>(static_cast<long>(blocks) * (blockIdx.y + 1) / splits);
  for (int b = lo + wave; b < hi; b += kWaves) {
    Oct xv[TF][4], wv[RF][4];
#pragma unroll
    for (int f = 0; f < TF; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i) xv[f][i] = load_oct_aligned(xr[f] + 128 * b + 32 * i);
#pragma unroll
    for (int f = 0; f < RF; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i) wv[f][i] = load_oct_aligned(wr[f] + 128 * b + 32 * i);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int f = 0; f < TF; ++f)
#pragma unroll
        for (int g = 0; g < RF; ++g) acc[f][g] = mfma<DT>(xv[f][i], wv[g][i], acc[f][g]);
  }
  if (wave > 0) {
#pragma unroll
    for (int f = 0; f < TF; ++f)
#pragma unroll
      for (int g = 0; g < RF; ++g) red[((wave - 1) * TF * RF + f * RF + g) * 64 + lane] = acc[f][g];
  }
  __syncthreads();
  if (wave > 0) return;
  float *out = part + (static_cast<size_t>(blockIdx.y) * M + tile.i0) * r;
#pragma unroll
  for (int f = 0; f < TF; ++f)
#pragma unroll
    for (int g = 0; g < RF; ++g) {
      float4_t v = acc[f][g];
#pragma unroll
      for (int w = 0; w < kWaves - 1; ++w) v += red[(w * TF * RF + f * RF + g) * 64 + lane];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * f + 4 * q + i, j = 16 * g + col;
        if (t < tile.n && j < r) out[static_cast<size_t>(t) * r + j] = v[i];
      }
    }
}

// ------------------------------------------------------------------ base + s h B^T

// y[t] = base[t] + s_a h_t B_a^T for a tile of tokens, kSpan = 256 columns a step (64 a
// wave); h_t the sum of the shares that the kernel above wrote, in two 16-bit
// pieces side by side along the instruction's k: 16 values of h and their rests
// against the same 16 values of B twice.
//
// D's rows are columns of y, in an order that leaves a lane eight neighbours:
// row 4 q + i of instruction m is column 8 q + 4 m + i.
constexpr int kSpan = 64 * kWaves;

template <int DT>
__device__ __forceinline__ void copy_row(const uint16_t *base, uint16_t *y, size_t row, int N, int n, int end) {
  // n: this thread's first column, eight a thread
  for (; n < end; n += 8 * kThreads) {
    const size_t at = row * N + n;
    if (n + 8 <= end) {
      store_oct(y + at, base ? load_oct(base + at) : Oct{{0, 0, 0, 0}});
    } else {
      for (int i = 0; i < end - n; ++i) y[at + i] = base ? base[at + i] : static_cast<uint16_t>(0);
    }
  }
}

template <int DT, int TF, int RC, bool BY_TOKEN, bool R8>
__global__ void __launch_bounds__(kThreads) adapters_expand_kernel(
    const float *__restrict__ part, int splits, int M, int N, int r, const uint16_t *__restrict__ B,
    const float *__restrict__ scales, int L, const int32_t *__restrict__ ids, const int32_t *__restrict__ offsets,
    const int32_t *__restrict__ perm, const uint16_t *base, uint16_t *y, float *__restrict__ h, int tiles, int steps) {
  constexpr int kRows = 16 * TF, kStride = 16 * RC + 4;
  __shared__ float hs[kRows * kStride];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
  const int from = blockIdx.y * steps * kSpan, end = min(from + steps * kSpan, N);
  Tile tile;
  if constexpr (BY_TOKEN) {
    const int t = blockIdx.x;
    tile = {adapter_of(ids, t, L), t, 1};
    if (tile.a < 0) {
      if (base != y) copy_row<DT>(base, y, t, N, from + 8 * threadIdx.x, end);
      if (h && blockIdx.y == 0)
        for (int j = threadIdx.x; j < r; j += kThreads) h[static_cast<size_t>(t) * r + j] = 0.f;
      return;
    }
  } else {
    if (static_cast<int>(blockIdx.x) >= tiles) {   // 64 tokens: those without an adapter
      const int t0 = (blockIdx.x - tiles) * 64;
      const uint64_t none = __ballot(t0 + lane < M && adapter_of(ids, min(t0 + lane, M - 1), L) < 0);
      for (uint64_t left = none; left; left &= left - 1) {
        const int t = t0 + __builtin_ctzll(left);
        if (base != y) copy_row<DT>(base, y, t, N, from + 8 * threadIdx.x, end);
        if (h && blockIdx.y == 0)
          for (int j = threadIdx.x; j < r; j += kThreads) h[static_cast<size_t>(t) * r + j] = 0.f;
      }
      return;
    }
    tile = tile_of(offsets, L, M, kRows, blockIdx.x);
    if (tile.a < 0) return;
  }
  // h of the tile's tokens; zeros in the columns past r and, so that nothing
  // unset is read, the rows past the last
  for (int i = threadIdx.x; i < kRows * 16 * RC; i += kThreads) {
    const int t = i / (16 * RC), j = i % (16 * RC);
    float v = 0.f;
    if (t < tile.n && j < r) {
      const float *p = part + static_cast<size_t>(tile.i0 + t) * r + j;
      for (int s = 0; s < splits; ++s) v += p[static_cast<size_t>(s) * M * r];
      if (h && blockIdx.y == 0) {
        const int at = BY_TOKEN ? tile.i0 : perm[tile.i0 + t];
        if (at >= 0 && at < M) h[static_cast<size_t>(at) * r + j] = v;
      }
    }
    hs[t * kStride + j] = v;
  }
  __syncthreads();
  Oct hv[TF][RC];
  float back[TF];
  size_t row[TF];
  bool live[TF];
  const float sa = scales[tile.a];
#pragma unroll
  for (int f = 0; f < TF; ++f) {
    const int t = 16 * f + col;
    int at = tile.i0 + min(t, tile.n - 1);
    if constexpr (!BY_TOKEN) at = perm[at];
    live[f] = t < tile.n && at >= 0 && at < M;
    row[f] = static_cast<size_t>(live[f] ? at : 0) * N;
    float v[RC][8], top = 0.f;
#pragma unroll
    for (int c = 0; c < RC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[c][i] = hs[t * kStride + 16 * c + 8 * (q & 1) + i];
        top = fmaxf(top, fabsf(v[c][i]));
      }
    top = fmaxf(top, __uint_as_float(xor_lane_u32<16>(__float_as_uint(top))));
    const Scale sc = scale_for<DT>(top);
    back[f] = sa * sc.back;
#pragma unroll
    for (int c = 0; c < RC; ++c) {
      Oct p[2];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] *= sc.to;
      split8<DT, 2>(v[c], p);
      hv[f][c] = q < 2 ? p[0] : p[1];
    }
  }
  const uint16_t *Ba = B + static_cast<size_t>(tile.a) * N * r;
  const size_t total = static_cast<size_t>(L) * N * r;
  for (int n0 = from + 64 * wave; n0 < end; n0 += kSpan) {
    Oct bv[4][RC];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int n = min(n0 + 32 * (m >> 1) + 8 * (col >> 2) + 4 * (m & 1) + (col & 3), N - 1);
#pragma unroll
      for (int c = 0; c < RC; ++c) {
        const int j = 16 * c + 8 * (q & 1);
        const size_t at = static_cast<size_t>(n) * r + j;
        if constexpr (R8) {
          bv[m][c] = j < r ? load_oct(Ba + at) : Oct{{0, 0, 0, 0}};
        } else {
          bv[m][c] = load_oct_part(Ba + at, r - j, total - min(total, static_cast<size_t>(tile.a) * N * r + at));
        }
      }
    }
    Oct yv[TF][2];
#pragma unroll
    for (int f = 0; f < TF; ++f)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int n = n0 + 32 * k + 8 * q;
        yv[f][k] = Oct{{0, 0, 0, 0}};
        if (base && live[f]) {
          if (n + 8 <= N) yv[f][k] = load_oct(base + row[f] + n);
          else yv[f][k] = load_oct_part(base + row[f] + n, N - n, 0);
        }
      }
#pragma unroll
    for (int f = 0; f < TF; ++f)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float4_t d[2] = {};
#pragma unroll
        for (int c = 0; c < RC; ++c)
#pragma unroll
          for (int m = 0; m < 2; ++m) d[m] = mfma<DT>(bv[2 * k + m][c], hv[f][c], d[m]);
        Oct o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4_t &v = d[i >> 1];
          const uint32_t b = yv[f][k].w[i];
          const float lo = fmaf(v[2 * (i & 1)], back[f], to_f32<DT>(static_cast<uint16_t>(b)));
          const float hi = fmaf(v[2 * (i & 1) + 1], back[f], to_f32<DT>(static_cast<uint16_t>(b >> 16)));
          o.w[i] = pack2<DT>(lo, hi);
        }
        const int n = n0 + 32 * k + 8 * q;
        if (live[f]) {
          if (n + 8 <= N) {
            store_oct(y + row[f] + n, o);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (n + i < N) y[row[f] + n + i] = static_cast<uint16_t>(o.w[i / 2] >> (16 * (i & 1)));
          }
        }
      }
  }
}

// How the forward pass is cut up.
struct ForwardPlan {
  bool by_token;
  int tf, rf;           // 16-token and 16-column pieces of a tile
  int tiles;            // at most
  int splits;           // shares of K
  int steps, chunks;    // kSpan-column steps of a workgroup, workgroups along N
};
constexpr int kFewTokens = 64;
constexpr int kWant = 1024;   // workgroups that fill the card

ForwardPlan forward_plan(const AdapterArgs &g, bool by_list) {
  ForwardPlan p{};
  p.by_token = !by_list;
  const int frags = (g.r + 15) / 16;
  p.rf = frags <= 1 ? 1 : frags <= 2 ? 2 : frags <= 4 ? 4 : 8;
  // tokens of an adapter on average decide the tile
  const int each = p.by_token ? 1 : g.M / std::max(1, std::min(g.L, g.M));
  p.tf = p.by_token || each <= 16 ? 1 : each <= 48 || p.rf >= 4 ? 2 : 4;
  const int rows = 16 * p.tf;
  p.tiles = p.by_token ? g.M : g.M / rows + std::min(g.L, g.M);
  const int likely = p.by_token ? g.M : std::max(1, g.M / rows);
  const int blocks = g.K / 128;
  // (the same for few tokens with and without an order: so is the result)
  const int cut = g.M <= kFewTokens ? std::max(1, g.M) : likely;
  p.splits = std::max(1, std::min({(kWant + cut - 1) / cut, (blocks + kWaves - 1) / kWaves, 16}));
  const int spans = (g.N + kSpan - 1) / kSpan;
  p.steps = std::max(1, std::min(8, static_cast<int>(static_cast<long>(spans) * likely / kWant)));
  p.chunks = (spans + p.steps - 1) / p.steps;
  return p;
}

template <int DT, int TF, int RC, bool BY_TOKEN>
void forward_go(const AdapterArgs &g, const ForwardPlan &p, hipStream_t s) {
  const uint16_t *x = static_cast<const uint16_t *>(g.x), *a = static_cast<const uint16_t *>(g.a);
  const uint16_t *b = static_cast<const uint16_t *>(g.b), *base = static_cast<const uint16_t *>(g.base);
  uint16_t *y = static_cast<uint16_t *>(g.y);
  float *part = static_cast<float *>(g.scratch);
  const dim3 block(kThreads);
  hipLaunchKernelGGL((adapters_shrink_kernel<DT, TF, RC, BY_TOKEN>), dim3(p.tiles, p.splits), block, 0, s, x, g.M, g.K,
                     g.r, a, g.L, g.ids, g.offsets, g.perm, part);
  const int others = BY_TOKEN || (base == y && !g.h) ? 0 : (g.M + 63) / 64;
  const dim3 grid(p.tiles + others, p.chunks);
  if (g.r % 8 == 0)
    hipLaunchKernelGGL((adapters_expand_kernel<DT, TF, RC, BY_TOKEN, true>), grid, block, 0, s, part, p.splits, g.M, g.N,
                       g.r, b, g.scales, g.L, g.ids, g.offsets, g.perm, base, y, g.h, p.tiles, p.steps);
  else
    hipLaunchKernelGGL((adapters_expand_kernel<DT, TF, RC, BY_TOKEN, false>), grid, block, 0, s, part, p.splits, g.M,
                       g.N, g.r, b, g.scales, g.L, g.ids, g.offsets, g.perm, base, y, g.h, p.tiles, p.steps);
}

template <int DT, int RC>
void forward_tiles(const AdapterArgs &g, const ForwardPlan &p, hipStream_t s) {
  if (p.by_token) return forward_go<DT, 1, RC, true>(g, p, s);
  if (p.tf == 1) return forward_go<DT, 1, RC, false>(g, p, s);
  if constexpr (RC < 4) {
    if (p.tf == 4) return forward_go<DT, 4, RC, false>(g, p, s);
  }
  forward_go<DT, 2, RC, false>(g, p, s);
}

template <int DT>
void forward_ranks(const AdapterArgs &g, const ForwardPlan &p, hipStream_t s) {
  if (p.rf == 1) forward_tiles<DT, 1>(g, p, s);
  else if (p.rf == 2) forward_tiles<DT, 2>(g, p, s);
  else if (p.rf == 4) forward_tiles<DT, 4>(g, p, s);
  else forward_tiles<DT, 8>(g, p, s);
}

}  // namespace

bool adapters_forward_by_list(const AdapterArgs &g) { return g.M > kFewTokens; }

size_t adapters_forward_ws_bytes(const AdapterArgs &g) {
  return static_cast<size_t>(g.M) * g.r * 4 * forward_plan(g, true).splits;
}

hipError_t launch_adapters_forward(const AdapterArgs &g, hipStream_t s) {
  const ForwardPlan p = forward_plan(g, g.offsets != nullptr);
  if (g.dtype == kF16) forward_ranks<kF16>(g, p, s);
  else forward_ranks<kBF16>(g, p, s);
  return hipGetLastError();
}

}  // namespace lbq
