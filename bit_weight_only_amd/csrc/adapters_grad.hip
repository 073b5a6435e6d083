// The adapters' gradients, with u_t = s_a dy_t B_a:
//
//   dB_a = s_a sum_t dy_t^T h_t      dx_t = base_t + u_t A_a      dA_a = sum_t u_t^T x_t
//
// dy and x are read once each. One pass over dy gives dB and, per 4 * 16 E columns, a
// share of u; one over x gives dA and dx. Between them the shares of u are added
// up and split into the 16-bit pieces that the matrix instructions take, once for
// all columns.
//
// A sum over tokens is a product whose long axis is the rows of dy or x: a lane
// loads E neighbours of eight rows and exchanges halves of registers, which gives
// it eight rows of each of its E columns, the operand of E instructions. Nothing
// goes through LDS.
#include "adapters.h"

#include <algorithm>

namespace lbq {

namespace {

using namespace adapters;

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kStep = 32;   // tokens of one step: the instruction's k

// Pieces of h and u in the sums over tokens, which stay fp32: as exact as fp32
// itself (two pieces of fp16 hold 22 bits, of bf16 only 16).
template <int DT>
constexpr int kPieces = DT == kF16 ? 2 : 3;

// A chunk: the tokens whose sums one workgroup keeps in registers.
struct Chunk {
  int a, i0, n;     // adapter, first list entry, tokens
  int step;         // number of its first step among all adapters'
  int slot;         // its place among the partial sums, -1: the adapter has one chunk
};

// Where an adapter with more than one chunk keeps a chunk's sums. Its chunks but
// the last are whole, so starts of two such lie `rows` apart, and so do two last
// ones: at most one of each kind starts in any `rows` entries.
__device__ __forceinline__ int slot_of(int i0, int rows, bool last) { return 2 * (i0 / rows) + (last ? 0 : 1); }

__device__ __forceinline__ void segment(const int32_t *offsets, int a, int M, int &lo, int &hi) {
  lo = min(max(offsets[a], 0), M);
  hi = min(max(offsets[a + 1], lo), M);
}

// Chunk number b of `rows` tokens each (a multiple of kStep), like tile_of. Offsets
// that are no sort's can name more steps than M tokens have (max_steps, what the
// workspace holds): a chunk with such a step is none.
__device__ __forceinline__ Chunk chunk_of(const int32_t *__restrict__ offsets, int L, int M, int rows, int max_steps,
                                          int b) {
  const int lane = threadIdx.x & 63;
  const int per = (L + 63) / 64;
  const int first = min(lane * per, L), last = min(first + per, L);
  int chunks = 0, steps = 0;
  for (int a = first; a < last; ++a) {
    int lo, hi;
    segment(offsets, a, M, lo, hi);
    chunks += (hi - lo + rows - 1) / rows;
    steps += (hi - lo + kStep - 1) / kStep;
  }
  int in_c = chunks, in_s = steps;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int c = __shfl_up(in_c, d), s = __shfl_up(in_s, d);
    if (lane >= d) {
      in_c += c;
      in_s += s;
    }
  }
  const uint64_t past = __ballot(in_c > b);
  if (past == 0) return {-1, 0, 0, 0, -1};
  const int owner = __builtin_ctzll(past);
  Chunk t{-1, 0, 0, 0, -1};
  if (lane == owner) {
    int at = in_c - chunks, step = in_s - steps;
    for (int a = first; a < last; ++a) {
      int lo, hi;
      segment(offsets, a, M, lo, hi);
      const int n = (hi - lo + rows - 1) / rows;
      if (b < at + n) {
        const int c = b - at, i0 = lo + c * rows;
        const int s0 = step + c * (rows / kStep), tokens = min(hi - i0, rows);
        if (s0 + (tokens + kStep - 1) / kStep <= max_steps)
          t = {a, i0, tokens, s0, n > 1 ? slot_of(i0, rows, c == n - 1) : -1};
        break;
      }
      at += n;
      step += (hi - lo + kStep - 1) / kStep;
    }
  }
  auto all = [&](int v) { return __builtin_amdgcn_readlane(v, owner); };
  return {all(t.a), all(t.i0), all(t.n), all(t.step), all(t.slot)};
}

// ------------------------------------------------------------------ pieces

// The operands that one step's tokens give, in the order in which lanes load them:
//   over  [steps][RF][pieces][64 lanes]: value 16 g + l % 16 of tokens 8 (l / 16) .. + 7,
//         times over_to[step]: the side of the sums over tokens;
//   along [steps][2][RF][64 lanes]: token 16 f + l % 16, its values 16 c + 8 (l / 16 % 2) ..
//         + 7, first pieces for l < 32 and second ones from there, times the token's
//         own power of two: the side of u A.
struct Pieces {
  Oct *over, *along;
  float *over_back, *along_back;   // [steps], [steps][kStep]: the inverse powers
};

// One workgroup per step: v[t][j] = scale * sum of `shares` shares (share s at src +
// s M r, rows by list entry), or the rows of h by token.
template <int DT, int RF, bool OF_H>
__global__ void __launch_bounds__(kThreads) adapters_pieces_kernel(const float *__restrict__ src, int shares, int M,
                                                                   int r, const float *__restrict__ scales, int L,
                                                                   const int32_t *__restrict__ offsets,
                                                                   const int32_t *__restrict__ perm, Pieces out) {
  constexpr int kP = kPieces<DT>, kCols = 16 * RF, kStride = kCols + 4;
  __shared__ float v[kStep * kStride];
  __shared__ float top[kWaves];
  const Chunk c = chunk_of(offsets, L, M, kStep, gridDim.x, blockIdx.x);
  if (c.a < 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
  const float sa = OF_H ? 1.f : scales[c.a];
  float m = 0.f;
  for (int i = threadIdx.x; i < kStep * kCols; i += kThreads) {
    const int t = i / kCols, j = i % kCols;
    float s = 0.f;
    if (t < c.n && j < r) {
      if constexpr (OF_H) {
        const int at = perm[c.i0 + t];
        if (at >= 0 && at < M) s = src[static_cast<size_t>(at) * r + j];
      } else {
        const float *p = src + static_cast<size_t>(c.i0 + t) * r + j;
        const size_t next = static_cast<size_t>(M) * r;
        int k = 0;
        for (; k + 8 <= shares; k += 8) {
          float w[8];
#pragma unroll
          for (int n = 0; n < 8; ++n) w[n] = p[(k + n) * next];
#pragma unroll
          for (int n = 0; n < 8; ++n) s += w[n];
        }
        for (; k < shares; ++k) s += p[k * next];
        s *= sa;
      }
    }
    v[t * kStride + j] = s;
    m = fmaxf(m, fabsf(s));
  }
  for (int d = 32; d > 0; d /= 2) m = fmaxf(m, __shfl_xor(m, d));
  if (lane == 0) top[wave] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) m = fmaxf(m, top[w]);
  const Scale sc = scale_for<DT>(m);
  if (threadIdx.x == 0) out.over_back[c.step] = sc.back;
  for (int g = wave; g < RF; g += kWaves) {
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = v[(8 * q + i) * kStride + 16 * g + col] * sc.to;
    Oct o[kP];
    split8<DT, kP>(w, o);
#pragma unroll
    for (int p = 0; p < kP; ++p) out.over[((static_cast<size_t>(c.step) * RF + g) * kP + p) * 64 + lane] = o[p];
  }
  if constexpr (!OF_H) {
    for (int f = wave; f < 2; f += kWaves) {
      const int t = 16 * f + col;
      float w[RF][8], mt = 0.f;
#pragma unroll
      for (int k = 0; k < RF; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          w[k][i] = v[t * kStride + 16 * k + 8 * (q & 1) + i];
          mt = fmaxf(mt, fabsf(w[k][i]));
        }
      mt = fmaxf(mt, __uint_as_float(xor_lane_u32<16>(__float_as_uint(mt))));
      const Scale st = scale_for<DT>(mt);
      if (q == 0) out.along_back[static_cast<size_t>(c.step) * kStep + t] = st.back;
#pragma unroll
      for (int k = 0; k < RF; ++k) {
        Oct o[2];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[k][i] *= st.to;
        split8<DT, 2>(w[k], o);
        out.along[((static_cast<size_t>(c.step) * 2 + f) * RF + k) * 64 + lane] = q < 2 ? o[0] : o[1];
      }
    }
  }
}

// ------------------------------------------------------------------ rows of dy and x

// E neighbouring values of eight rows: eight (16 bytes) or four.
template <int E>
struct Rows {
  uint32_t w[8][E / 2];
};

// Values E col .. of tokens 8 q + i of the step at list entry i0; end: columns there
// are in all (past it zeros).
template <int E>
__device__ __forceinline__ void load_rows(Rows<E> &v, const uint16_t *__restrict__ x, const size_t row[8], int n, int end) {
  struct __attribute__((packed, aligned(2))) Anywhere {
    uint32_t w[E / 2];
  };
  if (n + E <= end) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const Anywhere a = *reinterpret_cast<const Anywhere *>(x + row[i] + n);
#pragma unroll
      for (int d = 0; d < E / 2; ++d) v.w[i][d] = a.w[d];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int d = 0; d < E / 2; ++d) {
        uint32_t w = 0;
        if (n + 2 * d < end) w = x[row[i] + n + 2 * d];
        if (n + 2 * d + 1 < end) w |= static_cast<uint32_t>(x[row[i] + n + 2 * d + 1]) << 16;
        v.w[i][d] = w;
      }
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

__device__ __forceinline__ int token_at(const int32_t *perm, int i, int M) { return min(max(perm[min(i, M - 1)], 0), M - 1); }

// Sums of a chunk: v for (column n, value j) to the gradient [a][..] times scale, or to
// the partial sums [slot][..].
__device__ __forceinline__ void put(float *out, float *part, const Chunk &c, size_t size, size_t at, float v, float scale) {
  if (c.slot >= 0) part[static_cast<size_t>(c.slot) * size + at] = v;
  else out[static_cast<size_t>(c.a) * size + at] = v * scale;
}

// Zeros to a slice of the gradient of an adapter without tokens: columns n0 .. n1;
// value (n, j) at n * sn + j * sj.
__device__ __forceinline__ void clear(float *out, int r, int n0, int n1, size_t sn, size_t sj) {
  const int n = max(n1 - n0, 0);
  for (long i = threadIdx.x; i < static_cast<long>(n) * r; i += kThreads) {
    const int a = sn == 1 ? static_cast<int>(i / n) : static_cast<int>(i % r);
    const int b = sn == 1 ? static_cast<int>(i % n) : static_cast<int>(i / r);
    out[(n0 + b) * sn + a * sj] = 0.f;
  }
}

// ------------------------------------------------------------------ dy: dB and u

// Workgroup (chunk, slice): 16 E columns of dy a wavefront.
template <int DT, int E, int RF>
__global__ void __launch_bounds__(kThreads) adapters_dy_kernel(const uint16_t *__restrict__ dy, int M, int N, int r,
                                                               const uint16_t *__restrict__ B,
                                                               const float *__restrict__ scales, int L,
                                                               const int32_t *__restrict__ offsets,
                                                               const int32_t *__restrict__ perm, int rows, int chunks,
                                                               int max_steps, Pieces h, float *__restrict__ u_part,
                                                               float *__restrict__ dB, float *__restrict__ part) {
  constexpr int kP = kPieces<DT>, kCols = 16 * E, kSlice = kCols * kWaves, kK = kCols / 32;
  constexpr int kStride = 16 * RF + 1;
  __shared__ float red[2][kWaves][kStep * kStride];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
  if (static_cast<int>(blockIdx.x) >= chunks) {
    int lo, hi;
    const int a = blockIdx.x - chunks;
    segment(offsets, a, M, lo, hi);
    if (lo == hi)
      clear(dB + static_cast<size_t>(a) * N * r, r, blockIdx.y * kSlice, min(N, static_cast<int>(blockIdx.y + 1) * kSlice), r, 1);
    return;
  }
  const Chunk c = chunk_of(offsets, L, M, rows, max_steps, blockIdx.x);
  if (c.a < 0) return;
  const int n0 = blockIdx.y * kSlice + wave * kCols;
  // B of these columns: value 16 g + col of columns n0 + 32 k + 8 q .. + 7
  Oct bv[kK][RF];
  const uint16_t *Ba = B + static_cast<size_t>(c.a) * N * r;
#pragma unroll
  for (int k = 0; k < kK; ++k)
#pragma unroll
    for (int g = 0; g < RF; ++g) {
      const int j = 16 * g + col;
      uint32_t e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int n = n0 + 32 * k + 8 * q + i;
        e[i] = n < N && j < r ? Ba[static_cast<size_t>(n) * r + j] : 0;
      }
#pragma unroll
      for (int d = 0; d < 4; ++d) bv[k][g].w[d] = e[2 * d] | e[2 * d + 1] << 16;
    }
  float4_t acc[E][RF] = {};
  const int steps = (c.n + kStep - 1) / kStep;
  for (int s = 0; s < steps; ++s) {
    const int i0 = c.i0 + s * kStep, n = min(c.n - s * kStep, kStep);
    size_t row[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) row[i] = static_cast<size_t>(token_at(perm, i0 + min(8 * q + i, n - 1), M)) * N;
    Rows<E> v;
    load_rows<E>(v, dy, row, n0 + E * col, N);
    Oct a[2][kK];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const size_t at = static_cast<size_t>(token_at(perm, i0 + min(16 * f + col, n - 1), M)) * N;
#pragma unroll
      for (int k = 0; k < kK; ++k) {
        const int m = n0 + 32 * k + 8 * q;
        a[f][k] = m + 8 <= N ? load_oct(dy + at + m) : load_oct_part(dy + at + m, N - m, 0);
      }
    }
    Oct hv[RF][kP];
    const size_t step = c.step + s;
#pragma unroll
    for (int g = 0; g < RF; ++g)
#pragma unroll
      for (int p = 0; p < kP; ++p) hv[g][p] = h.over[((step * RF + g) * kP + p) * 64 + lane];
    // this wavefront's share of u
    float *mine = red[s & 1][wave];
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int g = 0; g < RF; ++g) {
        float4_t d = {};
#pragma unroll
        for (int k = 0; k < kK; ++k) d = mfma<DT>(a[f][k], bv[k][g], d);
#pragma unroll
        for (int i = 0; i < 4; ++i) mine[(16 * f + 4 * q + i) * kStride + 16 * g + col] = d[i];
      }
    if (n < kStep) drop_rows<E>(v, 8 * q, n);
    const float back = DT == kF16 ? h.over_back[step] : 1.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const Oct x = column<E>(v, e);
#pragma unroll
      for (int g = 0; g < RF; ++g) {
        if constexpr (DT == kF16) {
          float4_t d = {};
#pragma unroll
          for (int p = 0; p < kP; ++p) d = mfma<DT>(x, hv[g][p], d);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[e][g][i] = fmaf(d[i], back, acc[e][g][i]);
        } else {
#pragma unroll
          for (int p = 0; p < kP; ++p) acc[e][g] = mfma<DT>(x, hv[g][p], acc[e][g]);
        }
      }
    }
    // the slice's share of u (the other half of `red` is written next, so one
    // barrier a step is enough)
    __syncthreads();
    float *out = u_part + (static_cast<size_t>(blockIdx.y) * M + i0) * r;
    for (int i = threadIdx.x; i < n * r; i += kThreads) {
      const int t = i / r, j = i % r;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) sum += red[s & 1][w][t * kStride + j];
      out[i] = sum;
    }
  }
  const float sa = scales[c.a];
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int g = 0; g < RF; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = n0 + E * (4 * q + i) + e, j = 16 * g + col;
        if (n < N && j < r)
          put(dB, part, c, static_cast<size_t>(N) * r, static_cast<size_t>(n) * r + j, acc[e][g][i], sa);
      }
}

// ------------------------------------------------------------------ x: dA and dx

template <int DT, int E, int RF>
__global__ void __launch_bounds__(kThreads) adapters_x_kernel(const uint16_t *__restrict__ x, int M, int K, int r,
                                                              const uint16_t *__restrict__ A, int L,
                                                              const int32_t *__restrict__ ids,
                                                              const int32_t *__restrict__ offsets,
                                                              const int32_t *__restrict__ perm, int rows, int chunks,
                                                              int max_steps, Pieces u, const uint16_t *base, uint16_t *dx,
                                                              float *__restrict__ dA, float *__restrict__ part) {
  constexpr int kP = kPieces<DT>, kCols = 16 * E, kSlice = kCols * kWaves;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
  const int s0 = blockIdx.y * kSlice, s1 = min(K, s0 + kSlice);
  if (static_cast<int>(blockIdx.x) >= chunks + L) {   // 64 tokens: those without an adapter
    const int t0 = (blockIdx.x - chunks - L) * 64;
    int id = 0;
    if (t0 + lane < M) id = ids[t0 + lane];
    for (uint64_t left = __ballot(t0 + lane < M && (id < 0 || id >= L)); left; left &= left - 1) {
      const size_t at = static_cast<size_t>(t0 + __builtin_ctzll(left)) * K;
      for (int k = s0 + 8 * threadIdx.x; k < s1; k += 8 * kThreads)
        store_oct(dx + at + k, base ? load_oct_aligned(base + at + k) : Oct{{0, 0, 0, 0}});
    }
    return;
  }
  if (static_cast<int>(blockIdx.x) >= chunks) {
    int lo, hi;
    const int a = blockIdx.x - chunks;
    segment(offsets, a, M, lo, hi);
    if (lo == hi) clear(dA + static_cast<size_t>(a) * r * K, r, s0, s1, 1, K);
    return;
  }
  const Chunk c = chunk_of(offsets, L, M, rows, max_steps, blockIdx.x);
  if (c.a < 0) return;
  const int k0 = s0 + wave * kCols;
  if (k0 >= K) return;   // K is a multiple of 128, kCols of 64: all or nothing
  // A of these columns, transposed like the rows of x: column k0 + E col + e of
  // values 16 g + 8 (q % 2) .. + 7
  Oct av[E][RF];
  {
    const uint16_t *Aa = A + static_cast<size_t>(c.a) * r * K;
#pragma unroll
    for (int g = 0; g < RF; ++g) {
      size_t row[8];
      const int j = 16 * g + 8 * (q & 1);
#pragma unroll
      for (int i = 0; i < 8; ++i) row[i] = static_cast<size_t>(min(j + i, r - 1)) * K;
      Rows<E> v;
      load_rows<E>(v, Aa, row, k0 + E * col, K);
      drop_rows<E>(v, j, r);
#pragma unroll
      for (int e = 0; e < E; ++e) av[e][g] = column<E>(v, e);
    }
  }
  float4_t acc[E][RF] = {};
  const int steps = (c.n + kStep - 1) / kStep;
  for (int s = 0; s < steps; ++s) {
    const int i0 = c.i0 + s * kStep, n = min(c.n - s * kStep, kStep);
    const size_t step = c.step + s;
    size_t row[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) row[i] = static_cast<size_t>(token_at(perm, i0 + min(8 * q + i, n - 1), M)) * K;
    Rows<E> v;
    load_rows<E>(v, x, row, k0 + E * col, K);
    // dx: a lane holds columns k0 + 4 E q .. + 4 E - 1 of token 16 f + col
    Oct bv[2][E / 2];
    size_t at[2];
    bool live[2];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int t = perm[i0 + min(16 * f + col, n - 1)];
      live[f] = 16 * f + col < n && t >= 0 && t < M;
      at[f] = static_cast<size_t>(live[f] ? t : 0) * K + k0 + 4 * E * q;
#pragma unroll
      for (int k = 0; k < E / 2; ++k)
        bv[f][k] = base && live[f] ? load_oct_aligned(base + at[f] + 8 * k) : Oct{{0, 0, 0, 0}};
    }
    Oct uo[RF][kP], ua[2][RF];
#pragma unroll
    for (int g = 0; g < RF; ++g)
#pragma unroll
      for (int p = 0; p < kP; ++p) uo[g][p] = u.over[((step * RF + g) * kP + p) * 64 + lane];
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int g = 0; g < RF; ++g) ua[f][g] = u.along[((step * 2 + f) * RF + g) * 64 + lane];
    if (n < kStep) drop_rows<E>(v, 8 * q, n);
    const float back = DT == kF16 ? u.over_back[step] : 1.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const Oct xv = column<E>(v, e);
#pragma unroll
      for (int g = 0; g < RF; ++g) {
        if constexpr (DT == kF16) {
          float4_t d = {};
#pragma unroll
          for (int p = 0; p < kP; ++p) d = mfma<DT>(uo[g][p], xv, d);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[e][g][i] = fmaf(d[i], back, acc[e][g][i]);
        } else {
#pragma unroll
          for (int p = 0; p < kP; ++p) acc[e][g] = mfma<DT>(uo[g][p], xv, acc[e][g]);
        }
      }
    }
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      float4_t d[E] = {};
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int g = 0; g < RF; ++g) d[e] = mfma<DT>(av[e][g], ua[f][g], d[e]);
      const float tb = DT == kF16 ? u.along_back[step * kStep + 16 * f + col] : 1.f;
      if (!live[f]) continue;
      // column 4 E q + E i + e is d[e][i]
#pragma unroll
      for (int k = 0; k < E / 2; ++k) {
        Oct o;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int c0 = 8 * k + 2 * w;
          const uint32_t b = bv[f][k].w[w];
          o.w[w] = pack2<DT>(fmaf(d[c0 % E][c0 / E], tb, to_f32<DT>(static_cast<uint16_t>(b))),
                             fmaf(d[(c0 + 1) % E][(c0 + 1) / E], tb, to_f32<DT>(static_cast<uint16_t>(b >> 16))));
        }
        store_oct(dx + at[f] + 8 * k, o);
      }
    }
  }
#pragma unroll
  for (int g = 0; g < RF; ++g)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = 16 * g + 4 * q + i;
      if (j >= r) continue;
      const size_t at = static_cast<size_t>(j) * K + k0 + E * col;
      const size_t size = static_cast<size_t>(r) * K;
      float *out = c.slot >= 0 ? part + static_cast<size_t>(c.slot) * size : dA + static_cast<size_t>(c.a) * size;
#pragma unroll
      for (int e = 0; e < E; e += 4)
        *reinterpret_cast<float4_t *>(out + at + e) = float4_t{acc[e][g][i], acc[e + 1][g][i], acc[e + 2][g][i], acc[e + 3][g][i]};
    }
}

// The chunks' sums of the adapters that have several, added up in order.
__global__ void __launch_bounds__(kThreads) adapters_sum_kernel(const float *__restrict__ part, size_t size, int M,
                                                                const float *__restrict__ scales,
                                                                const int32_t *__restrict__ offsets, int rows,
                                                                float *__restrict__ out) {
  const int a = blockIdx.y;
  int lo, hi;
  segment(offsets, a, M, lo, hi);
  if (hi - lo <= rows) return;
  const float sa = scales ? scales[a] : 1.f;
  for (size_t i = static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x; i < size;
       i += static_cast<size_t>(gridDim.x) * kThreads) {
    float s = 0.f;
#pragma unroll 8
    for (int at = lo; at < hi; at += rows) s += part[static_cast<size_t>(slot_of(at, rows, hi - at <= rows)) * size + i];
    out[static_cast<size_t>(a) * size + i] = s * sa;
  }
}

// ------------------------------------------------------------------ plan

constexpr size_t kAlign = 256;
size_t round_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

struct Plan {
  int rf, e;
  int steps;                    // at most
  int rows_y, chunks_y, rows_x, chunks_x;
  int slices_y, slices_x;
  size_t over, along, over_back, along_back, u_part, sums, total;   // where in the workspace
};

// Tokens of a chunk: as many workgroups as fill the card, and chunks long enough
// that their sums' way through memory stays small beside the rows'.
int chunk_rows(int M, int slices) {
  constexpr int kWant = 512;
  const long rows = static_cast<long>(M) * slices / kWant;
  return static_cast<int>(std::min<long>(std::max<long>((rows + kStep - 1) / kStep * kStep, 128), 4096));
}

Plan plan_of(const AdapterArgs &g) {
  Plan p{};
  const int frags = (g.r + 15) / 16;
  p.rf = frags <= 1 ? 1 : frags <= 2 ? 2 : frags <= 4 ? 4 : 8;
  p.e = p.rf <= 2 ? 8 : 4;
  const int slice = 16 * p.e * kWaves;
  p.slices_y = (g.N + slice - 1) / slice;
  p.slices_x = (g.K + slice - 1) / slice;
  const int some = std::min(g.L, g.M);
  p.steps = g.M / kStep + some;
  p.rows_y = chunk_rows(g.M, p.slices_y);
  p.rows_x = chunk_rows(g.M, p.slices_x);
  p.chunks_y = g.M / p.rows_y + some;
  p.chunks_x = g.M / p.rows_x + some;
  const int pieces = g.dtype == kF16 ? 2 : 3;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round_up(bytes);
    return here;
  };
  p.over = take(static_cast<size_t>(p.steps) * p.rf * pieces * 64 * sizeof(Oct));
  p.along = take(static_cast<size_t>(p.steps) * 2 * p.rf * 64 * sizeof(Oct));
  p.over_back = take(static_cast<size_t>(p.steps) * 4);
  p.along_back = take(static_cast<size_t>(p.steps) * kStep * 4);
  p.u_part = take(static_cast<size_t>(p.slices_y) * g.M * g.r * 4);
  const size_t sums_y = g.M > p.rows_y ? 2 * (static_cast<size_t>(g.M) / p.rows_y + 1) * g.N * g.r * 4 : 0;
  const size_t sums_x = g.M > p.rows_x ? 2 * (static_cast<size_t>(g.M) / p.rows_x + 1) * g.K * g.r * 4 : 0;
  p.sums = take(std::max(sums_y, sums_x));   // dB's are done with when dA's begin
  p.total = at;
  return p;
}

template <int DT, int E, int RF>
void backward_go(const AdapterArgs &g, const Plan &p, hipStream_t s) {
  uint8_t *ws = static_cast<uint8_t *>(g.scratch);
  const Pieces q{reinterpret_cast<Oct *>(ws + p.over), reinterpret_cast<Oct *>(ws + p.along),
                 reinterpret_cast<float *>(ws + p.over_back), reinterpret_cast<float *>(ws + p.along_back)};
  float *u_part = reinterpret_cast<float *>(ws + p.u_part), *sums = reinterpret_cast<float *>(ws + p.sums);
  const uint16_t *a = static_cast<const uint16_t *>(g.a), *b = static_cast<const uint16_t *>(g.b);
  const uint16_t *base = static_cast<const uint16_t *>(g.base);
  uint16_t *dx = static_cast<uint16_t *>(g.y);
  const dim3 block(kThreads);
  auto sum = [&](size_t size, const float *scales, int rows, float *out) {
    const unsigned blocks = static_cast<unsigned>(std::min<size_t>((size + kThreads - 1) / kThreads, 2048));
    hipLaunchKernelGGL(adapters_sum_kernel, dim3(blocks, g.L), block, 0, s, sums, size, g.M, scales, g.offsets, rows, out);
  };
  if (p.steps > 0)
    hipLaunchKernelGGL((adapters_pieces_kernel<DT, RF, true>), dim3(p.steps), block, 0, s, g.h, 1, g.M, g.r, g.scales,
                       g.L, g.offsets, g.perm, q);
  hipLaunchKernelGGL((adapters_dy_kernel<DT, E, RF>), dim3(p.chunks_y + g.L, p.slices_y), block, 0, s,
                     static_cast<const uint16_t *>(g.dy), g.M, g.N, g.r, b, g.scales, g.L, g.offsets, g.perm, p.rows_y,
                     p.chunks_y, p.steps, q, u_part, g.d_b, sums);
  if (g.M > p.rows_y) sum(static_cast<size_t>(g.N) * g.r, g.scales, p.rows_y, g.d_b);
  if (p.steps > 0)
    hipLaunchKernelGGL((adapters_pieces_kernel<DT, RF, false>), dim3(p.steps), block, 0, s, u_part, p.slices_y, g.M, g.r,
                       g.scales, g.L, g.offsets, g.perm, q);
  const int others = base == dx ? 0 : (g.M + 63) / 64;
  hipLaunchKernelGGL((adapters_x_kernel<DT, E, RF>), dim3(p.chunks_x + g.L + others, p.slices_x), block, 0, s,
                     static_cast<const uint16_t *>(g.x), g.M, g.K, g.r, a, g.L, g.ids, g.offsets, g.perm, p.rows_x,
                     p.chunks_x, p.steps, q, base, dx, g.d_a, sums);
  if (g.M > p.rows_x) sum(static_cast<size_t>(g.K) * g.r, nullptr, p.rows_x, g.d_a);
}

template <int DT>
void backward_ranks(const AdapterArgs &g, const Plan &p, hipStream_t s) {
  if (p.rf == 1) backward_go<DT, 8, 1>(g, p, s);
  else if (p.rf == 2) backward_go<DT, 8, 2>(g, p, s);
  else if (p.rf == 4) backward_go<DT, 4, 4>(g, p, s);
  else backward_go<DT, 4, 8>(g, p, s);
}

}  // namespace

size_t adapters_backward_ws_bytes(const AdapterArgs &g) { return plan_of(g).total; }

hipError_t launch_adapters_backward(const AdapterArgs &g, hipStream_t s) {
  const Plan p = plan_of(g);
  if (g.dtype == kF16) backward_ranks<kF16>(g, p, s);
  else backward_ranks<kBF16>(g, p, s);
  return hipGetLastError();
}

}  // namespace lbq
