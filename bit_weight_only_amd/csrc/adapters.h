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
// loses no more than the second sum's own roundings (two pieces of fp16 2^-21 of it,
// three of bf16 2^-23).
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

// Pieces of a sum that enters another product.
template <int DT>
constexpr int kPieces = DT == kF16 ? 2 : 3;

// h (or u) as operands of a product with B (or A), whose operand c has values 16 c + 8
// (q % 2) .. + 7 in lanes q = lane / 16, so each of 16 values twice along the instruction's
// k: its first pieces meet the one, its second pieces the other. The third pieces of bf16 are
// operands of their own: of 32 values at once, where there are as many, against halves of
// two of the other side's operands.
template <int DT, int RC>
constexpr int kOperands = RC + (DT == kBF16 ? (RC + 1) / 2 : 0);
__host__ __device__ constexpr int operands_of(int dtype, int rc) { return rc + (dtype == kBF16 ? (rc + 1) / 2 : 0); }

// From a lane's eight values of each 16, as above.
template <int DT, int RC>
__device__ __forceinline__ void lay_operands(const float (&v)[RC][8], int q, Oct (&out)[kOperands<DT, RC>]) {
#pragma unroll
  for (int c = 0; c < RC; ++c) {
    Oct p[kPieces<DT>];
    split8<DT, kPieces<DT>>(v[c], p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      out[c].w[i] = q < 2 ? p[0].w[i] : p[1].w[i];
      if constexpr (DT == kBF16) {
        uint32_t &third = out[RC + c / 2].w[i];
        if (c % 2 == 0) third = q < 2 ? p[2].w[i] : 0u;
        else third = q < 2 ? third : p[2].w[i];
      }
    }
  }
}

// Operand k of the other side for operand k of h, k < kOperands.
template <int RC>
__device__ __forceinline__ Oct beside(const Oct (&b)[RC], int k, int q) {
  if (k < RC) return b[k];
  const int c = 2 * (k - RC);
  if (RC == 1) return b[0];   // (against zeros from q = 2 on)
  Oct o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.w[i] = q < 2 ? b[c].w[i] : b[RC == 1 ? 0 : c + 1].w[i];
  return o;
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

// E neighbouring values of R rows: eight (16 bytes) or four. Sixteen lanes hold 16 E
// neighbours of a row, so that a load's neighbouring lanes read neighbouring bytes:
// where they read different rows, as an operand's lanes do, the cache looks up 64
// places for the load and not 16 (470 MB through such loads and stores 111 us,
// 92 through a copy).
template <int E, int R = 8>
struct Rows {
  uint32_t w[R][E / 2];
};

template <int E, int R>
__device__ __forceinline__ void load_rows(Rows<E, R> &v, const uint16_t *x, const size_t (&row)[R], int n) {
  struct __attribute__((packed, aligned(2))) Anywhere {
    uint32_t w[E / 2];
  };
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const Anywhere a = *reinterpret_cast<const Anywhere *>(x + row[i] + n);
#pragma unroll
    for (int d = 0; d < E / 2; ++d) v.w[i][d] = a.w[d];
  }
}

// Column e of the eight rows.
template <int E>
__device__ __forceinline__ Oct column(const Rows<E> &v, int e) {
  const uint32_t sel = e & 1 ? 0x07060302u : 0x05040100u;
  Oct o;
#pragma unroll
  for (int d = 0; d < 4; ++d) o.w[d] = __builtin_amdgcn_perm(v.w[2 * d + 1][e / 2], v.w[2 * d][e / 2], sel);
  return o;
}

template <int E>
__device__ __forceinline__ void drop_rows(Rows<E> &v, int first, int n) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (first + i >= n) {
#pragma unroll
      for (int d = 0; d < E / 2; ++d) v.w[i][d] = 0;
    }
}

// out[row][n0 + E col ..] = base + back (P Q^T) for R = 4 tokens of a lane: d[e][i] is
// column e of token i. own: the first of the E columns that are this lane's and not
// its neighbour's (a piece that would reach past the last column starts earlier).
template <int DT, int E>
__device__ __forceinline__ void add_rows(uint16_t *out, const size_t (&row)[4], const bool (&live)[4], int n, int own,
                                         int end, const float4_t (&d)[E], const float4_t &back, const Rows<E, 4> &base) {
  struct __attribute__((packed, aligned(2))) Anywhere {
    uint32_t w[E / 2];
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (!live[i]) continue;
    Anywhere o;
#pragma unroll
    for (int w = 0; w < E / 2; ++w) {
      const uint32_t b = base.w[i][w];
      o.w[w] = pack2<DT>(fmaf(d[2 * w][i], back[i], to_f32<DT>(static_cast<uint16_t>(b))),
                         fmaf(d[2 * w + 1][i], back[i], to_f32<DT>(static_cast<uint16_t>(b >> 16))));
    }
    if (n + own + E <= end) {
      *reinterpret_cast<Anywhere *>(out + row[i] + n) = o;
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (e >= own && n + e < end) out[row[i] + n + e] = static_cast<uint16_t>(o.w[e / 2] >> (16 * (e & 1)));
    }
  }
}

// Tile number b of `rows` list entries each, adapter after adapter: its adapter
// (-1: past the last), first entry and count. One wavefront's lanes share the
// adapters; every lane gets the answer. Bad offsets give entries in [0, M) all
// the same.
struct Tile {
  int a, i0, n;
};
__device__ __forceinline__ void segment(const int32_t *__restrict__ offsets, int a, int M, int &lo, int &hi) {
  lo = min(max(offsets[a], 0), M);
  hi = min(max(offsets[a + 1], lo), M);
}
__device__ __forceinline__ int scan_lanes(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}
__device__ __forceinline__ Tile tile_of(const int32_t *__restrict__ offsets, int L, int M, int rows, int b) {
  const int lane = threadIdx.x & 63;
  const int per = (L + 63) / 64;
  const int first = min(lane * per, L), last = min(first + per, L);
  int lo = 0, hi = 0, tiles = 0;
  for (int a = first; a < last; ++a) {
    segment(offsets, a, M, lo, hi);
    tiles += (hi - lo + rows - 1) / rows;
  }
  const int incl = scan_lanes(tiles);
  const uint64_t past = __ballot(incl > b);
  if (past == 0) return {-1, 0, 0};
  const int owner = __builtin_ctzll(past);
  Tile t{-1, 0, 0};
  if (lane == owner) {
    int at = incl - tiles;
    for (int a = first; a < last; ++a) {
      if (per > 1) segment(offsets, a, M, lo, hi);
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

// A chunk: the tokens of one adapter that one workgroup goes through, in steps of
// `unit` tokens.
struct Chunk {
  int a, i0, n;     // adapter, first list entry, tokens
  int step;         // number of its first step among all adapters'
  int slot;         // its place among the partial sums, -1: the adapter has one chunk
};

// An adapter's tokens in chunks of at most `rows`, about equal and of whole steps.
struct Cut {
  int chunks, each;
};
__device__ __forceinline__ Cut cut_of(int tokens, int rows, int unit) {
  const int chunks = (tokens + rows - 1) / rows;
  return {chunks, chunks > 1 ? ((tokens + chunks - 1) / chunks + unit - 1) / unit * unit : rows};
}

// Where an adapter with more than one chunk keeps a chunk's sums. Its chunks but
// the last have over rows / 2 tokens, so that starts of two such lie that far
// apart, and so do two last ones: at most one of each kind starts in any
// rows / 2 entries.
__device__ __forceinline__ int slot_of(int i0, int rows, bool last) { return 2 * (i0 / (rows / 2)) + (last ? 0 : 1); }

// Chunk number b of up to `rows` tokens (a multiple of unit), like tile_of. Offsets
// that are no sort's can name more steps than M tokens have (max_steps, what the
// workspace holds): a chunk with such a step is none.
__device__ __forceinline__ Chunk chunk_of(const int32_t *__restrict__ offsets, int L, int M, int rows, int unit,
                                          int max_steps, int b) {
  const int lane = threadIdx.x & 63;
  const int per = (L + 63) / 64;
  const int first = min(lane * per, L), last = min(first + per, L);
  int lo = 0, hi = 0, chunks = 0, steps = 0;
  for (int a = first; a < last; ++a) {
    segment(offsets, a, M, lo, hi);
    chunks += (hi - lo + rows - 1) / rows;
    steps += (hi - lo + unit - 1) / unit;
  }
  const int in_c = scan_lanes(chunks), in_s = scan_lanes(steps);
  const uint64_t past = __ballot(in_c > b);
  if (past == 0) return {-1, 0, 0, 0, -1};
  const int owner = __builtin_ctzll(past);
  Chunk t{-1, 0, 0, 0, -1};
  if (lane == owner) {
    int at = in_c - chunks, step = in_s - steps;
    for (int a = first; a < last; ++a) {
      if (per > 1) segment(offsets, a, M, lo, hi);
      const Cut cut = cut_of(hi - lo, rows, unit);
      const int n = cut.chunks;
      if (b < at + n) {
        const int c = b - at, i0 = lo + c * cut.each;
        const int s0 = step + c * (cut.each / unit), tokens = min(hi - i0, cut.each);
        if (s0 + (tokens + unit - 1) / unit <= max_steps)
          t = {a, i0, max(tokens, 0), s0, n > 1 ? slot_of(i0, rows, c == n - 1) : -1};
        break;
      }
      at += n;
      step += (hi - lo + unit - 1) / unit;
    }
  }
  auto all = [&](int v) { return __builtin_amdgcn_readlane(v, owner); };
  return {all(t.a), all(t.i0), all(t.n), all(t.step), all(t.slot)};
}

// A chunk's tokens in LDS, -1 for what is none; up to a whole step the last once more.
// From there their numbers come without a wait for the loads that are under way, as
// a number that is loaded among them would.
constexpr int kMostTokens = 1024;
__device__ __forceinline__ void stage_tokens(const int32_t *__restrict__ perm, const Chunk &c, int unit, int M,
                                             int (&tokens)[kMostTokens]) {
  for (int i = threadIdx.x; i < (c.n + unit - 1) / unit * unit; i += blockDim.x) {
    const int t = perm[c.i0 + min(i, c.n - 1)];
    tokens[i] = t >= 0 && t < M ? t : -1;
  }
  __syncthreads();
}

// A few steps' values in turn: the next steps' loads are under way while a step is
// computed. They are always made, the last step's again at the end: a load in a
// branch would have the compiler wait for all that are under way.
// AHEAD: steps under way beside the one that is computed.
template <class V, int AHEAD = 1, class LOAD, class COMPUTE>
__device__ __forceinline__ void in_turn(int steps, LOAD load, COMPUTE compute) {
  V v[AHEAD + 1];
  if constexpr (AHEAD == 0) {
    for (int s = 0; s < steps; ++s) {
      load(v[0], s);
      compute(v[0], s);
    }
    return;
  }
  load(v[0], 0);
  if (steps == 1) return compute(v[0], 0);
#pragma unroll
  for (int i = 1; i < AHEAD; ++i) load(v[i], min(i, steps - 1));
  for (int s = 0;; s += AHEAD + 1) {
#pragma unroll
    for (int i = 0; i <= AHEAD; ++i) {
      load(v[(i + AHEAD) % (AHEAD + 1)], min(s + i + AHEAD, steps - 1));
      compute(v[i], s + i);
      if (s + i + 1 >= steps) return;
    }
  }
}

// Copies columns from .. end of the tokens t0 .. t0 + 63 that have no adapter from base
// (null: zeros) to y, rows of C; kThreads threads, eight columns and four rows of
// them under way each; the last eight may start earlier, and be some that are copied
// elsewhere too. `list` is LDS.
template <int kThreads>
__device__ __forceinline__ void copy_others(const int32_t *__restrict__ ids, int t0, int M, int L, const uint16_t *base,
                                            uint16_t *y, int C, int from, int end, int (&list)[64]) {
  const int lane = threadIdx.x & 63;
  int id = 0;
  if (t0 + lane < M) id = ids[t0 + lane];
  const uint64_t none = __ballot(t0 + lane < M && (id < 0 || id >= L));
  if (none == 0 || from >= end) return;
  if (threadIdx.x < 64 && (none >> lane & 1)) list[__builtin_popcountll(none & ((1ull << lane) - 1))] = t0 + lane;
  __syncthreads();
  const int units = (end - from + 7) / 8, total = __builtin_popcountll(none) * units;
  for (int u0 = threadIdx.x; u0 < total; u0 += 4 * kThreads) {
    Oct v[4];
    size_t at[4];
    int n[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int u = u0 + i * kThreads, c = max(min(from + u % units * 8, end - 8), 0);
      n[i] = u < total ? min(end - c, 8) : 0;
      at[i] = u < total ? static_cast<size_t>(list[u / units]) * C + c : 0;
      v[i] = Oct{{0, 0, 0, 0}};
      if (base && n[i] == 8) v[i] = load_oct(base + at[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (n[i] == 8) store_oct(y + at[i], v[i]);
      for (int k = 0; n[i] < 8 && k < n[i]; ++k) y[at[i] + k] = base ? base[at[i] + k] : static_cast<uint16_t>(0);
    }
  }
}

// Rows of fewer than eight values with zeros up to eight: the kernels read eight at a
// time.
constexpr int kNarrow = 8;
template <int kThreads>
__global__ void __launch_bounds__(kThreads) adapters_pad_kernel(const uint16_t *__restrict__ x, int M, int N,
                                                                uint16_t *__restrict__ out) {
  const int i = blockIdx.x * kThreads + threadIdx.x, t = i / kNarrow, n = i % kNarrow;
  if (t < M) out[i] = n < N ? x[t * N + n] : static_cast<uint16_t>(0);
}

}  // namespace adapters
}  // namespace lbq
