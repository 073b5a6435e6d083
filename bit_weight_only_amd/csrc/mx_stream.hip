// Products of MXFP4 tensors with few tokens: the weight is streamed once, the
// tokens stay in registers.
//
// A workgroup of eight waves splits K: wave w owns GPW 128-groups of every row
// and keeps the tokens' operands of its groups for its whole life, quantizing
// them itself where x comes in 16 bits (a lane holds one token's block of 32:
// its largest magnitude, its scale and its codes need no other lane). It then
// walks row tiles: NT tiles of 16 weight rows are loaded at once straight into
// operand registers (16 rows x 64 contiguous bytes per instruction), multiplied
// (v_mfma_scale_f32_16x16x128_f8f6f4), and the eight partial results are added
// in LDS in wave order.
//
// Operand layout: lane (r, q), r = lane & 15, q = lane >> 4, holds row r's block
// q of the 128-group and its scale byte; result register i of lane (c, q) is
// weight row 4 q + i, token c.
//
// Bound: HBM, (17/32) N K bytes; with fewer than a few MB to read, the latency
// of one load and the launch. One token 4096 -> 4096 5.2 us; 16 tokens 4096 ->
// 28672 15 us, 4.2 TB/s; 32 tokens on 136 of 256 experts of 2048 x 2048 57 us
// (304 MB fetched), 5.4 TB/s. Past 16 tokens: 32 4096 -> 28672 19 us, 64 23; 32
// 14336 -> 4096, which the tile kernel takes, 19.
#include "device.h"
#include "gemm_common.h"
#include "kernels.h"
#include "mxfp4.h"
#include "mx_tiles.h"

#include <algorithm>

namespace lbq {

namespace {

using namespace mxfp4;

constexpr int kWaves = 8, kThreads = 64 * kWaves;

// One block of 32 16-bit values as operand codes; returns the scale byte.
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
template <int DT>
__device__ __forceinline__ uint32_t quantize_block(const uint4 v[4], uint4 &codes) {
  const uint32_t w[16] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w,
                          v[2].x, v[2].y, v[2].z, v[2].w, v[3].x, v[3].y, v[3].z, v[3].w};
  u16x2_t m = __builtin_bit_cast(u16x2_t, w[0] & 0x7FFF7FFFu);
#pragma unroll
  for (int i = 1; i < 16; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, w[i] & 0x7FFF7FFFu));
  const uint32_t byte = scale_byte<DT>(m[0] > m[1] ? m[0] : m[1]);
  const float s = scale_value(byte);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = byte == 255u ? 0u : codes8<DT>(w + 4 * i, s);
  codes = make_uint4(c[0], c[1], c[2], c[3]);
  return byte;
}

__device__ __forceinline__ uint32_t lane_value(uint32_t v, int src) {
  return static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(src * 4, static_cast<int>(v)));
}

// Rows too long for the tokens' operands to stay in registers (GPW = 18: 90
// more a lane): LDS holds them, token t's codes at t (K / 2 + 16) bytes (the
// sixteen lanes of one read pass fall in sixteen 16-byte bank groups), its
// scale bytes behind all codes.
constexpr int kLongGroups = 18;
constexpr int kLongLds = 146 * 1024;
constexpr int long_lds_bytes(int K) { return 16 * (K / 2 + 16) + 16 * (K / 32); }

template <int MT, int GPW, int NT>
__global__ void __launch_bounds__(kThreads) mx_stream_kernel(MxGemm g, int T16, int walkers) {
  __shared__ __attribute__((aligned(16))) float4_t part[kWaves][NT * MT * 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // uniform: addresses by group in scalar registers
  const int r = lane & 15, q = lane >> 4;
  // `walkers` workgroups share a token tile and take its batches of rows in turn
  int i0, n_rows, e = 0, walker;
  if (g.E > 0) {
    const GroupTiles tiles(g.offsets, g.E, g.M, 16 * MT);
    const int id = xcd_order(blockIdx.x, tiles.total() * walkers);
    if (id < 0) return;
    const GroupTile t = tiles.find(id / walkers);
    walker = id % walkers;
    i0 = t.i0;
    n_rows = t.n;
    e = t.e;
  } else {
    i0 = blockIdx.x / walkers * (16 * MT);
    walker = blockIdx.x % walkers;
    n_rows = min(g.M - i0, 16 * MT);
  }
  const int G = g.K / kGroup, g0 = wave * GPW;
  const uint32_t row_bytes = g.K / 2;
  const size_t b_rows = g.E > 0 ? static_cast<size_t>(g.E) * g.N : g.N;

  // weight operands of tiles tb NT .. tb NT + NT - 1. Rows past N and groups
  // past G repeat the last one: the former are not stored, the latter meet
  // zero codes (and a NaN block there is a NaN block of the row anyway).
  uint4 w[NT][GPW];
  uint32_t ws[NT][GPW];
  auto load_weights = [&](int tb) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const size_t row = static_cast<size_t>(e) * g.N + min((tb * NT + t) * 16 + r, g.N - 1);
      const uint8_t *pc = static_cast<const uint8_t *>(g.b_codes) + row * row_bytes + 16 * q;
      const uint32_t sc = static_cast<uint32_t>(row);
#pragma unroll
      for (int i = 0; i < GPW; ++i) {
        const int gi = min(g0 + i, G - 1);
        w[t][i] = *reinterpret_cast<const uint4 *>(pc + 64 * gi);
        ws[t][i] = (static_cast<const uint32_t *>(g.b_scales) + static_cast<size_t>(gi) * b_rows)[sc];
      }
    }
  };
  int tb = walker;
  // the first weights travel while the tokens are quantized
  load_weights(tb);

  constexpr bool kLong = GPW == kLongGroups;
  static_assert(!kLong || MT == 1, "one token tile in LDS");
  __shared__ __attribute__((aligned(16))) uint8_t tok[kLong ? kLongLds : 16];
  const int tok_row = row_bytes + 16, tok_scales = 16 * tok_row, blocks = g.K / 32;
  if constexpr (kLong) {
    for (int u = tid; u < n_rows * blocks; u += kThreads) {
      const int t = u / blocks, b = u - t * blocks;
      int ia = i0 + t;
      if (g.perm) ia = g.perm[ia] / g.top_k;
      ia = min(max(ia, 0), g.a_rows - 1);
      uint4 codes;
      uint32_t byte;
      if (g.x) {
        const uint4 *px = reinterpret_cast<const uint4 *>(g.x) + (static_cast<size_t>(ia) * g.K + 32 * b) / 8;
        const uint4 v[4] = {px[0], px[1], px[2], px[3]};
        byte = g.dtype == kF16 ? quantize_block<kF16>(v, codes) : quantize_block<kBF16>(v, codes);
      } else {
        codes = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(g.a_codes) +
                                                 static_cast<size_t>(ia) * row_bytes + 16 * b);
        const uint32_t *words = static_cast<const uint32_t *>(g.a_scales) + static_cast<size_t>(b >> 2) * g.a_rows;
        byte = (words[ia] >> (8 * (b & 3))) & 0xFFu;
      }
      *reinterpret_cast<uint4 *>(tok + t * tok_row + 16 * b) = codes;
      tok[tok_scales + t * blocks + b] = static_cast<uint8_t>(byte);
    }
    barrier_lds();
  }

  // token operands in registers. Up to 8, 4, 2 or 1 tokens of a tile leave lanes without a
  // token of their own: those take further groups, 16 / span at a time, and hand
  // them on (one token on 14336 inputs: one block per lane instead of nine).
  uint4 a[MT][GPW];
  uint32_t as[MT][GPW];
  auto long_operand = [&](int i) {
    const int t = min(r, n_rows - 1), gi = min(g0 + i, G - 1);
    a[0][i] = *reinterpret_cast<const uint4 *>(tok + t * tok_row + 64 * gi + 16 * q);
    as[0][i] = tok[tok_scales + t * blocks + 4 * gi + q];
    if (g0 + i >= G) {
      a[0][i] = make_uint4(0, 0, 0, 0);
      as[0][i] = 127;
    }
  };
  const int span = MT > 1 || n_rows > 8 ? 16 : n_rows > 4 ? 8 : n_rows > 2 ? 4 : n_rows;
  const int per = 16 / span;   // groups per pass
#pragma unroll
  for (int m = 0; m < (kLong ? 0 : MT); ++m) {
    int ia = i0 + min(16 * m + (r & (span - 1)), n_rows - 1);
    if (g.perm) ia = g.perm[ia] / g.top_k;
    ia = min(max(ia, 0), g.a_rows - 1);
    uint4 codes{};
    uint32_t byte = 0;
#pragma unroll
    for (int i = 0; i < GPW; ++i) {
      if ((i & (per - 1)) == 0) {
        const int gi = min(g0 + i + r / span, G - 1);
        if (g.x) {
          const uint4 *px = reinterpret_cast<const uint4 *>(g.x) +
                            (static_cast<size_t>(ia) * g.K + kGroup * gi + 32 * q) / 8;
          const uint4 v[4] = {px[0], px[1], px[2], px[3]};
          byte = g.dtype == kF16 ? quantize_block<kF16>(v, codes) : quantize_block<kBF16>(v, codes);
        } else {
          codes = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(g.a_codes) +
                                                   static_cast<size_t>(ia) * row_bytes + 64 * gi + 16 * q);
          const uint32_t *words = static_cast<const uint32_t *>(g.a_scales) + static_cast<size_t>(gi) * g.a_rows;
          byte = (words[ia] >> (8 * q)) & 0xFFu;
        }
      }
      a[m][i] = codes;
      as[m][i] = byte;
      if (per > 1) {
        const int src = (lane & 48) | ((i & (per - 1)) * span + (r & (span - 1)));
        a[m][i] = make_uint4(lane_value(codes.x, src), lane_value(codes.y, src), lane_value(codes.z, src),
                             lane_value(codes.w, src));
        as[m][i] = lane_value(byte, src);
      }
      if (g0 + i >= G) {
        a[m][i] = make_uint4(0, 0, 0, 0);
        as[m][i] = 127;
      }
    }
  }

  for (;;) {
    float4_t acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[t][m] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < GPW; ++i) {
        if constexpr (kLong) long_operand(i);
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[t][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              operand(w[t][i]), operand(a[m][i]), acc[t][m], 4, 4, 0, static_cast<int>(ws[t][i] >> (8 * q)), 0,
              static_cast<int>(as[m][i]));
      }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int m = 0; m < MT; ++m) part[wave][(t * MT + m) * 64 + lane] = acc[t][m];
    const int cur = tb;
    tb += walkers;
    const bool more = static_cast<long>(tb) * NT < T16;
    if (more) load_weights(tb);   // in flight during the sums below
    barrier_lds();
    for (int v = tid; v < NT * MT * 64; v += kThreads) {
      float4_t sum = part[0][v];
#pragma unroll
      for (int k = 1; k < kWaves; ++k) sum += part[k][v];
      const int l = v & 63, tm = v >> 6, t = tm / MT, m = tm % MT;
      const int row = 16 * m + (l & 15), n = (cur * NT + t) * 16 + 4 * (l >> 4);
      if (row < n_rows) store4(g.y, g.dtype, (static_cast<size_t>(i0) + row) * g.N, n, g.N, sum);
    }
    if (!more) return;
    barrier_lds();   // the sums are read before the next ones are written
  }
}

// Dense: one workgroup per compute unit walks the row tiles, one tile of 16
// rows at a time (4096 -> 28672, one token: 14.0 us; two workgroups 15.7, two
// tiles at a time 16.0). Grouped: up to four per compute unit, since the grid
// holds slots for tiles that the routing may not fill, each with several tiles
// at a time (256 experts of 2048 x 2048, 32 tokens: 61 us; one workgroup per
// unit 107).
template <int MT, int GPW>
hipError_t launch(const MxGemm &g, int tiles, hipStream_t s) {
  constexpr int kMany = MT > 1 || GPW >= 8 ? 1 : GPW >= 4 ? 2 : 4;   // grouped calls come with MT = 1
  const int T16 = (g.N + 15) / 16;
  if (g.E > 0 && T16 >= 4 * kMany) {
    const int walkers = std::min((T16 + kMany - 1) / kMany, std::max(1, 1024 / tiles));
    hipLaunchKernelGGL((mx_stream_kernel<MT, GPW, kMany>), dim3(tiles * walkers), dim3(kThreads), 0, s, g, T16,
                       walkers);
  } else {
    const int walkers = std::min(T16, std::max(1, 256 / tiles));
    hipLaunchKernelGGL((mx_stream_kernel<MT, GPW, 1>), dim3(tiles * walkers), dim3(kThreads), 0, s, g, T16, walkers);
  }
  return hipGetLastError();
}

int groups_per_wave(int K) { return (K / kGroup + kWaves - 1) / kWaves; }

}  // namespace

bool mx_stream_supported(int rows, int K) {
  const int gpw = groups_per_wave(K);
  if (rows <= 16) return gpw <= 8 || (gpw <= kLongGroups && long_lds_bytes(K) <= kLongLds);
  return rows <= 32 ? gpw <= 8 : rows <= 64 && gpw <= 4;
}

hipError_t launch_mx_stream(const MxGemm &g, int rows, hipStream_t s) {
  const int mt = rows <= 16 ? 1 : rows <= 32 ? 2 : 4, gpw = groups_per_wave(g.K);
  const long n = (static_cast<long>(g.M) + 16 * mt - 1) / (16 * mt) + (g.E > 0 ? std::min(g.E, g.M) : 0);
  if (!mx_stream_supported(rows, g.K) || n > (1 << 24)) return hipErrorInvalidValue;
  const int tiles = static_cast<int>(n);
  if (mt == 1) {
    if (gpw <= 2) return launch<1, 2>(g, tiles, s);
    if (gpw <= 4) return launch<1, 4>(g, tiles, s);
    if (gpw <= 8) return launch<1, 8>(g, tiles, s);
    return launch<1, kLongGroups>(g, tiles, s);
  }
  if (mt == 2) {
    if (gpw <= 2) return launch<2, 2>(g, tiles, s);
    if (gpw <= 4) return launch<2, 4>(g, tiles, s);
    return launch<2, 8>(g, tiles, s);
  }
  if (gpw <= 2) return launch<4, 2>(g, tiles, s);
  return launch<4, 4>(g, tiles, s);
}

}  // namespace lbq
