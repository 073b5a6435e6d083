// Low-rank adapters of many requests beside a shared projection. Token t with
// adapter a = ids[t], scale s_a:
//
//   h_t = x_t A_a^T        y_t = base_t + s_a h_t B_a^T
//
// in two launches, or one; nothing uses atomics, so repeated calls give identical bits.
//
// The products are thin (r values): what bounds them is reading x and base and writing
// y, or, for few tokens, a load's latency and the launches. h stays fp32 between
// them.
#include "adapters.h"

#include <algorithm>
#include <type_traits>

namespace lbq {

namespace {

using namespace adapters;

constexpr int kThreads = 256, kWaves = kThreads / 64;

__device__ __forceinline__ int adapter_of(const int32_t *ids, int t, int L) {
  const int a = ids[t];
  return a >= 0 && a < L ? a : -1;
}

// Where eight values of h, and of a row of B, from j on are read: whole and inside
// the row. Of those read twice (below j) h gives zeros.
__device__ __forceinline__ int first_value(int j, int r) { return r > 8 && r % 8 != 0 ? min(j, r - 8) : j; }

// One lane's share of h as operands: values from j = 16 c + 8 (q % 2) on of a row of
// h in LDS, times a power of two of the token, whose inverse is `back`. Lane q's partner
// holds the row's other values.
template <int DT, int RC>
__device__ __forceinline__ void pieces_of(const float *row, int r, int q, Oct (&out)[kOperands<DT, RC>], float &back) {
  float v[RC][8], top = 0.f;
#pragma unroll
  for (int c = 0; c < RC; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int j = 16 * c + 8 * (q & 1), at = first_value(j, r) + i;
      v[c][i] = at >= j ? row[at] : 0.f;
      top = fmaxf(top, fabsf(v[c][i]));
    }
  top = fmaxf(top, __uint_as_float(xor_lane_u32<16>(__float_as_uint(top))));
  const Scale sc = scale_for<DT>(top);
  back = sc.back;
#pragma unroll
  for (int c = 0; c < RC; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] *= sc.to;
  lay_operands<DT, RC>(v, q, out);
}

// ------------------------------------------------------------------ x A^T

// 32 S values of 16 F rows on their way from memory through registers and LDS into
// operands: neighbouring lanes read neighbouring bytes (see Rows), which operands
// straight from memory do not. A row's 16-byte pieces lie in an order that keeps
// the banks apart.
template <int F, int S>
struct Staged {
  static constexpr int kPer = 4 * S, kRows = 64 / kPer, kLoads = 16 * F / kRows;   // pieces of a row, rows of a load
  Oct v[kLoads];
  template <class ROW>
  __device__ __forceinline__ void load(ROW row, int b) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) v[i] = load_oct_aligned(row(i) + 32 * S * b + 8 * (lane % kPer));
  }
  __device__ __forceinline__ void lay(uint16_t *lds) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int t = kRows * i + lane / kPer;
      *reinterpret_cast<uint4 *>(lds + (t * kPer + ((lane % kPer) ^ (t % kPer))) * 8) =
          make_uint4(v[i].w[0], v[i].w[1], v[i].w[2], v[i].w[3]);
    }
  }
  static __device__ __forceinline__ Oct operand(const uint16_t *lds, int f, int s) {
    const int lane = threadIdx.x & 63, t = 16 * f + (lane & 15);
    return load_oct_aligned(lds + (t * kPer + ((4 * s + (lane >> 4)) ^ (t % kPer))) * 8);
  }
};

// Between a wavefront's writes to LDS and its lanes' reads of one another's, and back. No
// instruction: a wavefront's accesses stay in order by themselves, if the compiler keeps
// them so. Of LDS alone: loads from memory stay under way.
__device__ __forceinline__ void lds_exchange() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local"); }

// The sums over blocks lo + wave, lo + wave + WAVES, .. below hi of a tile of up to
// 16 TF tokens and 16 RF values. Rows and values past the last are copies of the
// last (their results are dropped), so nothing is masked.
template <int TF, int RF, int S>
constexpr int kStage = (TF + RF) * 16 * 32 * S;   // LDS values of a wavefront
template <int DT, int TF, int RF, int S, int WAVES, bool BY_TOKEN>
__device__ __forceinline__ void shrink(const uint16_t *__restrict__ x, int M, int K, int r,
                                       const uint16_t *__restrict__ A, const int32_t *__restrict__ perm,
                                       const Tile &tile, int lo, int hi, uint16_t *lds, float4_t (&acc)[TF][RF]) {
  using X = Staged<TF, S>;
  using W = Staged<RF, S>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint16_t *xr[X::kLoads];
#pragma unroll
  for (int i = 0; i < X::kLoads; ++i) {
    int t = tile.i0 + min(X::kRows * i + lane / X::kPer, tile.n - 1);
    if constexpr (!BY_TOKEN) t = min(max(perm[t], 0), M - 1);
    xr[i] = x + static_cast<size_t>(t) * K;
  }
  const uint16_t *Aa = A + static_cast<size_t>(tile.a) * r * K;
  uint16_t *xl = lds + wave * kStage<TF, RF, S>, *wl = xl + TF * 16 * 32 * S;
#pragma unroll
  for (int f = 0; f < TF; ++f)
#pragma unroll
    for (int g = 0; g < RF; ++g) acc[f][g] = float4_t{0.f, 0.f, 0.f, 0.f};
  struct Block {
    X x;
    W w;
  };
  const int count = (hi - lo - wave + WAVES - 1) / WAVES;
  if (count <= 0) return;
  in_turn<Block>(
      count,
      [&](Block &v, int i) {
        const int b = lo + wave + i * WAVES;
        v.x.load([&](int n) { return xr[n]; }, b);
        v.w.load([&](int n) { return Aa + static_cast<size_t>(min(W::kRows * n + lane / W::kPer, r - 1)) * K; }, b);
      },
      [&](const Block &v, int) {
        v.x.lay(xl);
        v.w.lay(wl);
        lds_exchange();
#pragma unroll
        for (int s = 0; s < S; ++s) {
          Oct a[TF];
#pragma unroll
          for (int f = 0; f < TF; ++f) a[f] = X::operand(xl, f, s);
#pragma unroll
          for (int g = 0; g < RF; ++g) {
            const Oct w = W::operand(wl, g, s);
#pragma unroll
            for (int f = 0; f < TF; ++f) acc[f][g] = mfma<DT>(a[f], w, acc[f][g]);
          }
        }
        lds_exchange();   // the next block's values go to the same place
      });
}

// The waves' sums added up; value j of token t to put(t, j, v).
template <int TF, int RF, int WAVES, class F>
__device__ __forceinline__ void join(const float4_t (&acc)[TF][RF], float4_t *red, F put) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int f = 0; f < TF; ++f)
#pragma unroll
    for (int g = 0; g < RF; ++g) red[((wave * TF + f) * RF + g) * 64 + lane] = acc[f][g];
  __syncthreads();
  for (int u = threadIdx.x; u < TF * RF * 64; u += 64 * WAVES) {
    float4_t v = red[u];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += red[w * TF * RF * 64 + u];
    const int f = u / (RF * 64), g = u / 64 % RF, l = u % 64;
#pragma unroll
    for (int i = 0; i < 4; ++i) put(16 * f + 4 * (l >> 4) + i, 16 * g + (l & 15), v[i]);
  }
}

// Few tokens: part[s][row][j] = the sum over the s-th share of K, a tile per
// workgroup column. BY_TOKEN: every token is a tile of its own, and a row its
// number; else rows are list entries. Bound by latency (64 tokens on 64 adapters of 4096
// columns, rank 16: 5.0 us for 9 MB), which is why K is cut up until there are about
// 512 workgroups, with at most kMostShares shares, that the next launch reads at once.
template <int DT, int RF, bool BY_TOKEN>
__global__ void __launch_bounds__(kThreads) adapters_shares_kernel(const uint16_t *__restrict__ x, int M, int K, int r,
                                                                   const uint16_t *__restrict__ A, int L,
                                                                   const int32_t *__restrict__ ids,
                                                                   const int32_t *__restrict__ offsets,
                                                                   const int32_t *__restrict__ perm,
                                                                   float *__restrict__ part) {
  constexpr int kS = RF == 8 ? 2 : 4;
  constexpr size_t kLds = std::max(sizeof(float4_t) * kWaves * RF * 64, sizeof(uint16_t) * kWaves * kStage<1, RF, kS>);
  __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];
  Tile tile;
  if constexpr (BY_TOKEN) tile = {adapter_of(ids, blockIdx.x, L), static_cast<int>(blockIdx.x), 1};
  else tile = tile_of(offsets, L, M, 16, blockIdx.x);
  if (tile.a < 0) return;
  const int blocks = K / (32 * kS), splits = gridDim.y;
  const int lo = static_cast<int>(static_cast<long>(blocks) * blockIdx.y / splits);
  const int hi = static_cast<int>(static_cast<long>(blocks) * (blockIdx.y + 1) / splits);
  float4_t acc[1][RF];
  shrink<DT, 1, RF, kS, kWaves, BY_TOKEN>(x, M, K, r, A, perm, tile, lo, hi, reinterpret_cast<uint16_t *>(lds), acc);
  __syncthreads();
  float4_t *red = reinterpret_cast<float4_t *>(lds);
  float *out = part + (static_cast<size_t>(blockIdx.y) * M + tile.i0) * r;
  join<1, RF, kWaves>(acc, red, [&](int t, int j, float v) {
    if (t < tile.n && j < r) out[static_cast<size_t>(t) * r + j] = v;
  });
}

// Many tokens, bound by reading x (8192 tokens of 14336, rank 8: 235 MB in 47.0 us, 5.0
// TB/s; 1777 tokens of 5120, rank 64: 19.0 us, 71 workgroups' latency): a workgroup
// takes a tile's whole K, and leaves h as the operands
// that the second product loads: pieces[(tile TF + f) kOperands + k][lane], back[tile 16 TF + t].
// Shares of K with their sums made in the second product, once per 2048 columns, cost
// more than they gave (1777 tokens, 5120 -> 17408, rank 64: both kernels 134 us).
constexpr int kManyThreads = 512;
template <int DT, int TF, int RF>
__global__ void __launch_bounds__(kManyThreads) adapters_h_kernel(const uint16_t *__restrict__ x, int M, int K, int r,
                                                                  const uint16_t *__restrict__ A, int L,
                                                                  const int32_t *__restrict__ offsets,
                                                                  const int32_t *__restrict__ perm,
                                                                  Oct *__restrict__ pieces, float *__restrict__ back,
                                                                  float *__restrict__ h) {
  constexpr int kW = kManyThreads / 64, kStride = 16 * RF + 4, kS = RF >= 4 ? 2 : 4;
  constexpr size_t kLds = std::max(sizeof(float4_t) * kW * TF * RF * 64, sizeof(uint16_t) * kW * kStage<TF, RF, kS>);
  __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];
  __shared__ float hs[16 * TF * kStride];
  const Tile tile = tile_of(offsets, L, M, 16 * TF, blockIdx.x);
  if (tile.a < 0) return;
  float4_t acc[TF][RF];
  shrink<DT, TF, RF, kS, kW, false>(x, M, K, r, A, perm, tile, 0, K / (32 * kS), reinterpret_cast<uint16_t *>(lds), acc);
  __syncthreads();
  float4_t *red = reinterpret_cast<float4_t *>(lds);
  join<TF, RF, kW>(acc, red, [&](int t, int j, float v) { hs[t * kStride + j] = t < tile.n && j < r ? v : 0.f; });
  __syncthreads();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (wave < TF) {
    Oct o[kOperands<DT, RF>];
    float b;
    pieces_of<DT, RF>(hs + (16 * wave + (lane & 15)) * kStride, r, lane >> 4, o, b);
    const size_t at = static_cast<size_t>(blockIdx.x) * TF + wave;
#pragma unroll
    for (int k = 0; k < kOperands<DT, RF>; ++k) pieces[(at * kOperands<DT, RF> + k) * 64 + lane] = o[k];
    if (lane < 16) back[16 * at + lane] = b;
  }
  if (h)
    for (int i = threadIdx.x; i < 16 * TF * 16 * RF; i += kManyThreads) {
      const int t = i / (16 * RF), j = i % (16 * RF);
      if (t < tile.n && j < r) {
        const int token = perm[tile.i0 + t];
        if (token >= 0 && token < M) h[static_cast<size_t>(token) * r + j] = hs[t * kStride + j];
      }
    }
}

// ------------------------------------------------------------------ base + s h B^T

// y[t] = base[t] + s_a h_t B_a^T for a tile of tokens, kSpan = 256 columns a step (64 a
// wave); h_t in 16-bit pieces (see kOperands).
//
// D's rows are columns of y, in an order that leaves a lane eight neighbours:
// row 4 q + i of instruction m is column 8 q + 4 m + i. A piece of eight columns, or
// of eight values of B, that would reach past the last starts earlier, so that
// every load is whole and none is in a branch; what it has twice is not stored, or
// meets a zero of h.
constexpr int kSpan = 64 * kWaves, kMostShares = 16;

// RANK: kWhole, r a multiple of 8; kMore, above 8; kLess, below (single loads).
enum { kWhole, kMore, kLess };

// A row of B as an operand's share: values from 16 c + 8 (q % 2) on.
template <int RC, int RANK>
__device__ __forceinline__ void load_weights(Oct (&b)[RC], const uint16_t *__restrict__ row, int r) {
  const int q = threadIdx.x >> 4 & 3;
#pragma unroll
  for (int c = 0; c < RC; ++c) {
    const int j = 16 * c + 8 * (q & 1);
    if constexpr (RANK == kLess) {
      uint32_t e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        e[i] = row[min(j + i, r - 1)];
        e[i] = j + i < r ? e[i] : 0;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) b[c].w[i] = e[2 * i] | e[2 * i + 1] << 16;
    } else {
      // (past r all of h's values are zeros, and B's from here its own)
      b[c] = load_oct(row + min(j, r - 8));
    }
  }
}

// The 64 columns from n0 of 16 tokens: base + back (h B^T), stored to the token's row
// `to` where it is live. y: base's values, 32 columns each.
template <int DT, int RC>
__device__ __forceinline__ void add_product(const Oct (&b)[4][RC], const Oct (&hv)[kOperands<DT, RC>], float back, const Oct (&y)[2],
                                            uint16_t *to, bool live, int n0, int N, int width) {
  const int q = threadIdx.x >> 4 & 3;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float4_t d[2] = {};
#pragma unroll
    for (int c = 0; c < kOperands<DT, RC>; ++c)
#pragma unroll
      for (int m = 0; m < 2; ++m) d[m] = mfma<DT>(beside(b[2 * k + m], c, q), hv[c], d[m]);
    Oct o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4_t &z = d[i >> 1];
      const uint32_t v = y[k].w[i];
      o.w[i] = pack2<DT>(fmaf(z[2 * (i & 1)], back, to_f32<DT>(static_cast<uint16_t>(v))),
                         fmaf(z[2 * (i & 1) + 1], back, to_f32<DT>(static_cast<uint16_t>(v >> 16))));
    }
    const int n = n0 + 32 * k + 8 * q;
    if (!live) continue;
    if (n + 8 <= N) {
      store_oct(to + n, o);
    } else {
      const int first = min(n, width - 8);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (first + i >= n && first + i < N) to[first + i] = static_cast<uint16_t>(o.w[i / 2] >> (16 * (i & 1)));
    }
  }
}

// base's values of the 64 columns from n0; null: zeros.
__device__ __forceinline__ void load_base(Oct (&y)[2], const uint16_t *base, size_t row, int n0, int width) {
  const int q = threadIdx.x >> 4 & 3;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    y[k] = Oct{{0, 0, 0, 0}};
    if (base) y[k] = load_oct(base + row * width + min(n0 + 32 * k + 8 * q, width - 8));
  }
}

// The tokens t0 .. t0 + 63 without an adapter: y = base, h = 0.
__device__ __forceinline__ void others(const int32_t *ids, int t0, int M, int L, int N, int r, const uint16_t *base,
                                       uint16_t *y, float *h, int from, int end) {
  __shared__ int list[64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (h && from == 0) {
    const uint64_t none = __ballot(t0 + lane < M && adapter_of(ids, min(t0 + lane, M - 1), L) < 0);
    for (int t = wave; t < 64; t += kWaves)
      if (none >> t & 1)
        for (int j = lane; j < r; j += 64) h[static_cast<size_t>(t0 + t) * r + j] = 0.f;
  }
  if (base != y) copy_others<kThreads>(ids, t0, M, L, base, y, N, from, end, list);
}

// Few tokens: one tile of up to 16 a workgroup column, bound by reading B (64 tokens on
// 64 adapters, 28672 columns, rank 16: 12.9 us, 4.5 TB/s) or, for a few tokens, by
// latency (one token, 4096 columns 6.2 us in one launch). FROM: h is the sum of the shares,
// by token or by list entry, or (by token) is made here, by every workgroup for
// itself: one launch less, for A's way to each of them from the caches (kOneBytes).
enum { kByToken, kByEntry, kOneLaunch };
template <int DT, int RC, int FROM, int RANK>
__global__ void __launch_bounds__(FROM == kOneLaunch ? kManyThreads : kThreads) adapters_few_kernel(
    const uint16_t *__restrict__ x, int K, const uint16_t *__restrict__ A, const float *__restrict__ part, int splits, int M, int N, int r, const uint16_t *__restrict__ B,
    const float *__restrict__ scales, int L, const int32_t *__restrict__ ids, const int32_t *__restrict__ offsets,
    const int32_t *__restrict__ perm, const uint16_t *base, const uint16_t *rows_of_base, uint16_t *y,
    float *__restrict__ h, int tiles, int steps) {
  constexpr int kStride = 16 * RC + 4, kMine = FROM == kOneLaunch ? kManyThreads : kThreads, kW = kMine / 64;
  constexpr int kSpan = 64 * kW;
  constexpr bool BY_TOKEN = FROM != kByEntry;
  __shared__ float hs[16 * kStride];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
  const int from = blockIdx.y * steps * kSpan, end = min(from + steps * kSpan, N);
  Tile tile;
  if constexpr (BY_TOKEN) {
    const int t = blockIdx.x;
    tile = {adapter_of(ids, t, L), t, 1};
    if (tile.a < 0) {
      for (int n = from + threadIdx.x; base != y && n < end; n += kMine)
        y[static_cast<size_t>(t) * N + n] = base ? base[static_cast<size_t>(t) * N + n] : static_cast<uint16_t>(0);
      if (h && blockIdx.y == 0)
        for (int j = threadIdx.x; j < r; j += kMine) h[static_cast<size_t>(t) * r + j] = 0.f;
      return;
    }
  } else {
    if (static_cast<int>(blockIdx.x) >= tiles)
      return others(ids, (blockIdx.x - tiles) * 64, M, L, N, r, base, y, h, from, end);
    tile = tile_of(offsets, L, M, 16, blockIdx.x);
    if (tile.a < 0) return;
  }
  const int width = max(N, kNarrow);   // columns of a row of rows_of_base
  int token = tile.i0 + min(col, tile.n - 1);
  if constexpr (!BY_TOKEN) token = perm[token];
  const bool live = col < tile.n && token >= 0 && token < M;
  const size_t row = static_cast<size_t>(min(max(token, 0), M - 1));
  if constexpr (FROM == kOneLaunch) {
    constexpr int kS = RC >= 4 ? 2 : 4;
    constexpr size_t kLds = std::max(sizeof(float4_t) * kW * RC * 64, sizeof(uint16_t) * kW * kStage<1, RC, kS>);
    __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];
    float4_t acc[1][RC];
    shrink<DT, 1, RC, kS, kW, true>(x, M, K, r, A, perm, tile, 0, K / (32 * kS), reinterpret_cast<uint16_t *>(lds), acc);
    __syncthreads();
    join<1, RC, kW>(acc, reinterpret_cast<float4_t *>(lds), [&](int t, int j, float v) {
      hs[t * kStride + j] = j < r ? v : 0.f;   // (the one token sixteen times)
      if (h && blockIdx.y == 0 && t == 0 && j < r) h[static_cast<size_t>(tile.i0) * r + j] = v;
    });
  } else {
    // the shares added up; zeros past r and, so that nothing unset is read, past the
    // tile's last token
    for (int i = threadIdx.x; i < 16 * 16 * RC; i += kThreads) {
      const int t = i / (16 * RC), j = i % (16 * RC);
      float v = 0.f;
      if (t < tile.n && j < r) {
        const float *p = part + static_cast<size_t>(tile.i0 + t) * r + j;
        float w[kMostShares];   // all under way at once
#pragma unroll
        for (int s = 0; s < kMostShares; ++s) w[s] = s < splits ? p[static_cast<size_t>(s) * M * r] : 0.f;
#pragma unroll
        for (int s = 0; s < kMostShares; ++s) v += w[s];
        if (h && blockIdx.y == 0) {
          const int at = BY_TOKEN ? tile.i0 : perm[tile.i0 + t];
          if (at >= 0 && at < M) h[static_cast<size_t>(at) * r + j] = v;
        }
      }
      hs[t * kStride + j] = v;
    }
  }
  __syncthreads();
  Oct hv[kOperands<DT, RC>];
  float back;
  pieces_of<DT, RC>(hs + col * kStride, r, q, hv, back);
  back *= scales[tile.a];
  const uint16_t *Ba = B + static_cast<size_t>(tile.a) * N * r;
  struct Step {
    Oct b[4][RC], y[2];
  };
  const int n0 = from + 64 * wave, count = (end - n0 + kSpan - 1) / kSpan;
  if (n0 < end)
    in_turn<Step>(
        count,
        [&](Step &v, int s) {
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const int n = min(n0 + s * kSpan + 32 * (m >> 1) + 8 * (col >> 2), width - 8) + 4 * (m & 1) + (col & 3);
            load_weights<RC, RANK>(v.b[m], Ba + static_cast<size_t>(min(n, N - 1)) * r, r);
          }
          load_base(v.y, base ? rows_of_base : nullptr, row, n0 + s * kSpan, width);
        },
        [&](const Step &v, int s) {
          add_product<DT, RC>(v.b, hv, back, v.y, y + row * N, live, n0 + s * kSpan, N, width);
        });
}

// Many tokens: a wavefront takes 16 E columns, whose part of B stays in registers,
// and goes through a chunk of an adapter's tokens, 16 TF a step. D's rows are tokens,
// so that a lane holds E neighbouring columns of four of them. UNIT: tokens of the
// tiles in which h's operands were made. Slices of columns are neighbours in the grid, so
// that rows are read and written whole by workgroups that run together. Bound by
// HBM: 8192 tokens, 14336 columns, rank 16, bf16 91 us for 470 MB, 5.2 TB/s (with two pieces of
// h, which lose bits where base and h B^T cancel, 87); rank 64, 146 us, 3.2, of which the
// matrix cores' part no longer hides (with two pieces 119).
template <int DT, int E, int TF, int RC, int RANK>
__global__ void __launch_bounds__(kThreads, RC <= 4 ? 2 : 1) adapters_y_kernel(
    const Oct *__restrict__ pieces, const float *__restrict__ backs, int unit, int M, int N, int r,
    const uint16_t *__restrict__ B, const float *__restrict__ scales, int L, const int32_t *__restrict__ ids,
    const int32_t *__restrict__ offsets, const int32_t *__restrict__ perm, const uint16_t *base,
    const uint16_t *rows_of_base, uint16_t *y, float *__restrict__ h, int rows, int chunks, int max_steps) {
  constexpr int kStep = 16 * TF, kColumns = 16 * E;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
  const int from = blockIdx.x * kColumns * kWaves;
  if (static_cast<int>(blockIdx.y) >= chunks)
    return others(ids, (blockIdx.y - chunks) * 64, M, L, N, r, base, y, h, from, min(from + kColumns * kWaves, N));
  const Chunk c = chunk_of(offsets, L, M, rows, unit, max_steps, blockIdx.y);
  const int n0 = from + kColumns * wave;
  if (c.a < 0) return;
  __shared__ __attribute__((aligned(16))) int tokens[kMostTokens];
  stage_tokens(perm, c, kStep, M, tokens);
  if (n0 >= N) return;
  const int width = max(N, kNarrow);   // columns of a row of rows_of_base
  // columns n .. n + E - 1, of which those from n + own on are this lane's
  const int n = min(n0 + E * col, width - E), own = n0 + E * col - n;
  Oct b[E][RC];
#pragma unroll
  for (int e = 0; e < E; ++e) load_weights<RC, RANK>(b[e], B + (static_cast<size_t>(c.a) * N + min(n + e, N - 1)) * r, r);
  const float sa = scales[c.a];
  constexpr int kOps = kOperands<DT, RC>;
  struct Step {
    Oct h[TF][kOps];
    Rows<E, 4> y[TF];
    float4_t back[TF];
  };
  // (a step ahead costs more registers than there are from rank 33 on: 8192 tokens, rank
  // 64, 14336 columns, both launches with it fp16 155 and bf16 255 us, without 141 and 165)
  constexpr int kAhead = RC >= 4 ? 0 : 1;
  in_turn<Step, kAhead>(
      (c.n + kStep - 1) / kStep,
      [&](Step &v, int s) {
#pragma unroll
        for (int f = 0; f < TF; ++f) {
          // (a chunk's steps are whole but for the last, whose second half may be none)
          const size_t at = static_cast<size_t>(c.step) * (unit / 16) + min(s * TF + f, (c.n - 1) / 16);
          if (base) {
            size_t row[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              row[i] = static_cast<size_t>(max(tokens[s * kStep + 16 * f + 4 * q + i], 0)) * width;
            load_rows(v.y[f], rows_of_base, row, n);
          } else {
            v.y[f] = Rows<E, 4>{};
          }
          v.back[f] = *reinterpret_cast<const float4_t *>(backs + 16 * at + 4 * q);
#pragma unroll
          for (int k = 0; k < kOps; ++k) v.h[f][k] = pieces[(at * kOps + k) * 64 + lane];
        }
      },
      [&](const Step &v, int s) {
#pragma unroll
        for (int f = 0; f < TF; ++f) {
          float4_t d[E] = {};
#pragma unroll
          for (int k = 0; k < kOps; ++k)
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] = mfma<DT>(v.h[f][k], beside(b[e], k, q), d[e]);
          size_t row[4];
          bool live[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = s * kStep + 16 * f + 4 * q + i, to = tokens[t];
            live[i] = t < c.n && to >= 0;
            row[i] = static_cast<size_t>(max(to, 0)) * N;
          }
          add_rows<DT, E>(y, row, live, n, own, N, d, v.back[f] * sa, v.y[f]);
        }
      });
}

// ------------------------------------------------------------------ plan

// How the forward pass is cut up.
struct ForwardPlan {
  bool few, by_token, one;
  int tf, rf;           // 16-token and 16-value pieces of a tile
  int e;                // many tokens: columns of a lane
  int tiles;            // at most
  int splits;           // shares of K
  int steps;            // kSpan-column steps of a workgroup
  int rows, chunks;     // many tokens: of a chunk, at most
  size_t pieces, back, pad, total;   // where in the workspace (part at its start)
};
// up to so many tokens a call has no sort and no operands laid out between its launches
constexpr int kFewTokens = 64;
// A's bytes that a workgroup reads to make h for itself, and such workgroups, at most.
// Called one by one, one launch saves what the other costs the caller (4096 -> 4096, rank 16, 1 to
// 32 tokens 7.3 us against 11.8, 64 tokens 8.3 and 11.5). From a graph the two are equal up to 32
// tokens (6.0), then A's reads count: 64 tokens 8.6 and 7.7, 16 tokens of 8192 columns 8.1 and
// 6.1. At both limits at once one launch is the slower either way (64 tokens of 2048 columns,
// rank 64, 21.4 and 20.1, 22.6 and 20.7).
constexpr long kOneBytes = 256 << 10, kOneGroups = 512;

ForwardPlan forward_plan(const AdapterArgs &g, bool by_list) {
  ForwardPlan p{};
  p.few = g.M <= kFewTokens;
  p.by_token = !by_list;
  const int frags = (g.r + 15) / 16;
  p.rf = frags <= 1 ? 1 : frags <= 2 ? 2 : frags <= 4 ? 4 : 8;
  const int some = std::max(1, std::min(g.L, g.M));
  // tokens of an adapter on average decide the tile: two pieces of 16 tokens share A's
  // operands, where they would not mostly be empty (rank above 64: registers)
  p.tf = p.few || g.M / some <= 16 || p.rf == 8 ? 1 : 2;
  const int unit = 16 * p.tf, spans = (g.N + kSpan - 1) / kSpan;
  p.e = p.rf <= 2 ? 8 : 4;
  if (p.few) {
    // (the same with and without an order: so is the result)
    p.splits = std::max(1, std::min({512 / std::max(1, g.M), (g.K / 128 + kWaves - 1) / kWaves, kMostShares}));
    p.steps = std::max(1, std::min(8, static_cast<int>(static_cast<long>(spans) * g.M / 512)));
    p.one = p.rf < 8 && static_cast<long>(p.rf) * 32 * g.K <= kOneBytes && static_cast<long>(g.M) * ((spans + 1) / 2) <= kOneGroups;
    if (p.one) {
      p.by_token = true;
      p.steps = 1;
    }
  } else {
    // chunks so long that 1024 workgroups have one each, but at least 128 tokens (4000
    // tokens of 96 adapters, 2048 columns 13.6 us, with 32 18.9), or 32 where that is
    // still no more than a workgroup a compute unit (257 tokens, 2047 columns 16.2 us with
    // 128, 11.0 with 32; both launches of 500 tokens, 8 adapters, 4096 columns 18.8 and 14.4;
    // of 1000 tokens, 32 adapters, 14336 columns 25.4 and 27.5)
    const long groups = (g.N + 64 * p.e - 1) / (64 * p.e), rows = g.M * groups / 1024;
    const long least = (g.M / 32 + some) * groups <= 256 ? 32 : 128;
    p.rows = static_cast<int>(std::min(std::max((rows + 31) / 32 * 32, least), static_cast<long>(kMostTokens)));
    p.chunks = g.M / p.rows + some;
  }
  p.tiles = p.few && p.by_token ? g.M : g.M / unit + some;
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  if (!p.few) {
    p.back = up(static_cast<size_t>(p.tiles) * p.tf * operands_of(g.dtype, p.rf) * 64 * sizeof(Oct));
    p.pad = p.back + up(static_cast<size_t>(p.tiles) * unit * 4);
  } else {
    p.pad = p.one ? 0 : up(static_cast<size_t>(p.splits) * g.M * g.r * 4);
  }
  p.total = p.pad + (g.N < kNarrow ? static_cast<size_t>(g.M) * kNarrow * 2 : 0);
  return p;
}

template <int DT, int RC>
void forward_rank(const AdapterArgs &g, const ForwardPlan &p, hipStream_t s) {
  const uint16_t *x = static_cast<const uint16_t *>(g.x), *a = static_cast<const uint16_t *>(g.a);
  const uint16_t *b = static_cast<const uint16_t *>(g.b), *base = static_cast<const uint16_t *>(g.base);
  uint16_t *y = static_cast<uint16_t *>(g.y);
  uint8_t *ws = static_cast<uint8_t *>(g.scratch);
  const dim3 block(kThreads);
  const uint16_t *wide = base;
  if (base && g.N < kNarrow) {
    uint16_t *pad = reinterpret_cast<uint16_t *>(ws + p.pad);
    hipLaunchKernelGGL(adapters_pad_kernel<kThreads>, dim3((g.M * kNarrow + kThreads - 1) / kThreads), block, 0, s, base,
                       g.M, g.N, pad);
    wide = pad;
  }
  const unsigned spans = (g.N + kSpan - 1) / kSpan, rest = base == y && !g.h ? 0 : (g.M + 63) / 64;
  const int rank = g.r % 8 == 0 ? kWhole : g.r > 8 ? kMore : kLess;
  if (p.few) {
    float *part = reinterpret_cast<float *>(ws);
    auto go = [&](auto first, auto second, bool by_token) {
      hipLaunchKernelGGL(first, dim3(p.tiles, p.splits), block, 0, s, x, g.M, g.K, g.r, a, g.L, g.ids, g.offsets,
                         g.perm, part);
      hipLaunchKernelGGL(second, dim3(p.tiles + (by_token ? 0 : rest), (spans + p.steps - 1) / p.steps), block, 0, s, x,
                         g.K, a, part, p.splits, g.M, g.N, g.r, b, g.scales, g.L, g.ids, g.offsets, g.perm, base, wide, y, g.h,
                         p.tiles, p.steps);
    };
    auto pick = [&](auto by_token) {
      constexpr bool kBy = decltype(by_token)::value;
      constexpr int kFrom = kBy ? kByToken : kByEntry;
      auto first = adapters_shares_kernel<DT, RC, kBy>;
      if (rank == kWhole) go(first, adapters_few_kernel<DT, RC, kFrom, kWhole>, kBy);
      else if (rank == kMore) go(first, adapters_few_kernel<DT, RC, kFrom, kMore>, kBy);
      else if constexpr (RC == 1) go(first, adapters_few_kernel<DT, RC, kFrom, kLess>, kBy);
    };
    if constexpr (RC < 8) {
      auto once = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(g.M, (spans + 1) / 2), dim3(kManyThreads), 0, s, x, g.K, a, nullptr, 0, g.M, g.N,
                           g.r, b, g.scales, g.L, g.ids, nullptr, nullptr, base, wide, y, g.h, 0, 1);
      };
      if (p.one) {
        if (rank == kWhole) once(adapters_few_kernel<DT, RC, kOneLaunch, kWhole>);
        else if (rank == kMore) once(adapters_few_kernel<DT, RC, kOneLaunch, kMore>);
        else if constexpr (RC == 1) once(adapters_few_kernel<DT, RC, kOneLaunch, kLess>);
        return;
      }
    }
    if (p.by_token) pick(std::true_type{});
    else pick(std::false_type{});
    return;
  }
  Oct *pieces = reinterpret_cast<Oct *>(ws);
  float *back = reinterpret_cast<float *>(ws + p.back);
  auto go = [&](auto first, auto second) {
    hipLaunchKernelGGL(first, dim3(p.tiles), dim3(kManyThreads), 0, s, x, g.M, g.K, g.r, a, g.L, g.offsets, g.perm,
                       pieces, back, g.h);
    hipLaunchKernelGGL(second, dim3((g.N + 64 * p.e - 1) / (64 * p.e), p.chunks + rest), block, 0, s, pieces, back,
                       16 * p.tf, g.M, g.N, g.r, b, g.scales, g.L, g.ids, g.offsets, g.perm, base, wide, y, g.h, p.rows,
                       p.chunks, p.tiles);
  };
  auto pick = [&](auto tf) {
    // two pieces of 16 tokens a step where the registers allow it (bf16 up to rank 16, whose
    // third pieces take some: 8192 tokens, 4096 columns, both launches with two 83 us, with one 79;
    // rank 64, 2000 tokens, 14336 columns with two 49, with one 55)
    constexpr bool kTwo = RC == 4 || (RC == 1 && DT == kF16);
    constexpr int kTF = kTwo ? decltype(tf)::value : 1, kE = RC <= 2 ? 8 : 4;
    auto first = adapters_h_kernel<DT, decltype(tf)::value, RC>;
    if (rank == kWhole) go(first, adapters_y_kernel<DT, kE, kTF, RC, kWhole>);
    else if (rank == kMore) go(first, adapters_y_kernel<DT, kE, kTF, RC, kMore>);
    else if constexpr (RC == 1) go(first, adapters_y_kernel<DT, kE, kTF, RC, kLess>);
  };
  if constexpr (RC < 8) {
    if (p.tf == 2) return pick(std::integral_constant<int, 2>{});
  }
  pick(std::integral_constant<int, 1>{});
}

template <int DT>
void forward_ranks(const AdapterArgs &g, const ForwardPlan &p, hipStream_t s) {
  if (p.rf == 1) forward_rank<DT, 1>(g, p, s);
  else if (p.rf == 2) forward_rank<DT, 2>(g, p, s);
  else if (p.rf == 4) forward_rank<DT, 4>(g, p, s);
  else forward_rank<DT, 8>(g, p, s);
}

}  // namespace

bool adapters_forward_by_list(const AdapterArgs &g) { return g.M > kFewTokens; }

size_t adapters_forward_ws_bytes(const AdapterArgs &g) { return forward_plan(g, true).total; }

hipError_t launch_adapters_forward(const AdapterArgs &g, hipStream_t s) {
  const ForwardPlan p = forward_plan(g, g.offsets != nullptr);
  if (g.dtype == kF16) forward_ranks<kF16>(g, p, s);
  else forward_ranks<kBF16>(g, p, s);
  return hipGetLastError();
}

}  // namespace lbq
