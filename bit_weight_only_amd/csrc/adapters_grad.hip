// The adapters' gradients, with u_t = s_a dy_t B_a:
//
//   dB_a = s_a sum_t dy_t^T h_t      dx_t = base_t + u_t A_a      dA_a = sum_t u_t^T x_t
//
// dy and x are read once each. One pass over dy gives dB and, per 512 columns, a share
// of u; one over x gives dA and dx. Between them the shares of u are added
// up and split into the 16-bit pieces that the matrix instructions take, once for
// all columns.
//
// A sum over tokens is a product whose long axis is the rows of dy or x: a lane
// loads E neighbours of eight rows and exchanges halves of registers, which gives
// it eight rows of each of its E columns, the operand of E instructions.
//
// What bounds them is dy, x and dx, read and written once (8192 tokens, 4096 -> 14336,
// rank 16, bf16: 437 MB with dx's base, 144 us for all six launches).
#include "adapters.h"

#include <algorithm>

namespace lbq {

namespace {

using namespace adapters;

constexpr int kThreads = 256, kWaves = kThreads / 64;       // of the pass over x and the sums
// of the pass over dy, by pieces of 16 values: as many columns share a u as fit LDS
constexpr int dy_waves(int rf) { return rf == 8 ? 4 : 8; }
constexpr int kE = 4;                                        // columns of a lane in both
constexpr int kPieceThreads = 512;
constexpr int kStep = 32;   // tokens of one step: the instruction's k

// ------------------------------------------------------------------ pieces

// The operands that one step's tokens give, in the order in which lanes load them:
//   over  [steps][RF][pieces][64 lanes]: value 16 g + l % 16 of tokens 8 (l / 16) .. + 7,
//         times a power of two of the step's value: the side of the sums over tokens (a
//         value's tokens meet one another only, so that small values lose nothing beside
//         large ones);
//   along [steps][2][kOperands][64 lanes]: token 16 f + l % 16, its values as operands of a
//         product along them, times the token's own power of two: the side of u A.
struct Pieces {
  Oct *over, *along;
  float *over_back, *along_back;   // [steps][16 RF], [steps][kStep]: the inverse powers
};

// Bound by latency (256 steps at rank 16 4.7 us for h, 6.3 for the 28 shares of u; rank 64
// 7.7 and 14.6). One workgroup per step: v[t][j] = scale * sum of `shares` shares (share s at src +
// s M r, rows by list entry), or the rows of h by token.
template <int DT, int RF, bool OF_H>
__global__ void __launch_bounds__(kPieceThreads) adapters_pieces_kernel(const float *__restrict__ src, int shares, int M,
                                                                   int r, const float *__restrict__ scales, int L,
                                                                   const int32_t *__restrict__ offsets,
                                                                   const int32_t *__restrict__ perm, Pieces out) {
  constexpr int kP = kPieces<DT>, kCols = 16 * RF, kStride = kCols + 4;
  __shared__ float v[kStep * kStride];
  const Chunk c = chunk_of(offsets, L, M, kStep, kStep, gridDim.x, blockIdx.x);
  if (c.a < 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
  const float sa = OF_H ? 1.f : scales[c.a];
  for (int i = threadIdx.x; i < kStep * kCols; i += kPieceThreads) {
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
        for (; k < shares; k += 16) {   // sixteen under way
          float w[16];
#pragma unroll
          for (int n = 0; n < 16; ++n) w[n] = k + n < shares ? p[(k + n) * next] : 0.f;
#pragma unroll
          for (int n = 0; n < 16; ++n) s += w[n];
        }
        s *= sa;
      }
    }
    v[t * kStride + j] = s;
  }
  __syncthreads();
  for (int g = wave; g < RF; g += kPieceThreads / 64) {
    float w[8], m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = v[(8 * q + i) * kStride + 16 * g + col];
      m = fmaxf(m, fabsf(w[i]));
    }
    m = fmaxf(m, __uint_as_float(xor_lane_u32<16>(__float_as_uint(m))));
    m = fmaxf(m, __uint_as_float(xor_lane_u32<32>(__float_as_uint(m))));
    const Scale sc = scale_for<DT>(m);
    if (q == 0) out.over_back[static_cast<size_t>(c.step) * kCols + 16 * g + col] = sc.back;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] *= sc.to;
    Oct o[kP];
    split8<DT, kP>(w, o);
#pragma unroll
    for (int p = 0; p < kP; ++p) out.over[((static_cast<size_t>(c.step) * RF + g) * kP + p) * 64 + lane] = o[p];
  }
  if constexpr (!OF_H) {
    for (int f = wave; f < 2; f += kPieceThreads / 64) {
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
      for (int k = 0; k < RF; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) w[k][i] *= st.to;
      Oct o[kOperands<DT, RF>];
      lay_operands<DT, RF>(w, q, o);
#pragma unroll
      for (int k = 0; k < kOperands<DT, RF>; ++k)
        out.along[((static_cast<size_t>(c.step) * 2 + f) * kOperands<DT, RF> + k) * 64 + lane] = o[k];
    }
  }
}

// Sums of a chunk: v for (column n, value j) to the gradient [a][..] times scale, or to
// the partial sums [slot][..].
__device__ __forceinline__ void put(float *out, float *part, const Chunk &c, size_t size, size_t at, float v, float scale) {
  if (c.slot >= 0) part[static_cast<size_t>(c.slot) * size + at] = v;
  else out[static_cast<size_t>(c.a) * size + at] = v * scale;
}

// `count` zeros, by a workgroup.
template <int kThreads>
__device__ __forceinline__ void clear(float *out, size_t count) {
  struct __attribute__((packed, aligned(4))) Four {
    float v[4];
  };
  for (size_t i = 4 * threadIdx.x; i < count; i += 4 * kThreads) {
    if (i + 4 <= count) *reinterpret_cast<Four *>(out + i) = Four{{0.f, 0.f, 0.f, 0.f}};
    else
      for (size_t k = i; k < count; ++k) out[k] = 0.f;
  }
}

// ------------------------------------------------------------------ dy: dB and u

// The operands of a step (COUNT loads of 64 lanes) on their way through registers into
// LDS, where all wavefronts read them.
template <int COUNT, int WAVES>
struct Shared {
  static constexpr int kEach = (COUNT + WAVES - 1) / WAVES;
  typedef uint32_t vec_t __attribute__((ext_vector_type(4)));
  vec_t v[kEach];
  __device__ __forceinline__ void load(const Oct *from) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      v[i] = reinterpret_cast<const vec_t *>(from)[min(wave + i * WAVES, COUNT - 1) * 64 + lane];
  }
  __device__ __forceinline__ void lay(Oct *lds) const {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (wave + i * WAVES < COUNT) reinterpret_cast<vec_t *>(lds)[(wave + i * WAVES) * 64 + lane] = v[i];
  }
};

// A barrier that orders LDS alone, and leaves the loads under way.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Workgroup (chunk, slice): 16 E columns of dy a wavefront. width: columns of a row
// of dy, N or, where that is less, 8. A piece of columns that would reach past
// the last starts earlier, so that every load is whole and none is in a branch;
// what it has twice is not stored, or meets a zero of B.
//
// dy's values lie by rows for the sums over tokens; for u they go through LDS, 16-byte
// pieces of a row in an order that keeps the banks apart.
//
// Two sums over different axes from one read: 8192 tokens, 14336 columns 75 us at rank
// 16 (3.1 TB/s; waiting between the barriers), 168 at rank 64 (matrix cores 23 % busy,
// a third of it for h's three pieces, and one workgroup a compute unit). A second read
// in a kernel of its own would be 44 us more.
template <int DT, int RF>
__global__ void __launch_bounds__(64 * dy_waves(RF), RF == 1 ? 4 : RF <= 4 ? 2 : 1) adapters_dy_kernel(
    const uint16_t *__restrict__ dy, int width, int M, int N, int r, const uint16_t *__restrict__ B,
    const float *__restrict__ scales, int L, const int32_t *__restrict__ offsets, const int32_t *__restrict__ perm,
    int rows, int chunks, int max_steps, Pieces h, float *__restrict__ u_part, float *__restrict__ dB,
    float *__restrict__ part) {
  constexpr int kDyWaves = dy_waves(RF), kDyThreads = 64 * kDyWaves;
  constexpr int E = kE, kP = kPieces<DT>, kCols = 16 * E, kSlice = kCols * kDyWaves, kK = kCols / 32;
  constexpr int kStride = 16 * RF + 1;
  __shared__ float red[kDyWaves][kStep * kStride];
  __shared__ __attribute__((aligned(16))) uint16_t tile[kDyWaves][kStep * kCols];
  __shared__ Oct hs[RF * kP * 64];
  __shared__ float backs[16 * RF];
  __shared__ __attribute__((aligned(16))) int tokens[kMostTokens];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
  if (static_cast<int>(blockIdx.y) >= chunks) {
    int lo, hi;
    const int a = blockIdx.y - chunks;
    segment(offsets, a, M, lo, hi);
    const int n0 = blockIdx.x * kSlice, n1 = min(N, n0 + kSlice);   // (no tokens: zeros)
    if (lo == hi) clear<kDyThreads>(dB + (static_cast<size_t>(a) * N + n0) * r, static_cast<size_t>(n1 - n0) * r);
    return;
  }
  const Chunk c = chunk_of(offsets, L, M, rows, kStep, max_steps, blockIdx.y);
  if (c.a < 0) return;
  const int n0 = blockIdx.x * kSlice + wave * kCols;
  stage_tokens(perm, c, kStep, M, tokens);
  // B of these columns: value 16 g + col of the columns that lie at 32 k + 8 q .. + 7 of
  // a row in LDS, zero for those that lie there twice or are none
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
        const int at = 32 * k + 8 * q + i, m = n0 + at / E * E, n = min(m, width - E) + at % E;
        e[i] = Ba[static_cast<size_t>(min(n, N - 1)) * r + min(j, r - 1)];
        e[i] = n >= m && n < N && j < r ? e[i] : 0;
      }
#pragma unroll
      for (int d = 0; d < 4; ++d) bv[k][g].w[d] = e[2 * d] | e[2 * d + 1] << 16;
    }
  constexpr int kAhead = 1;
  float4_t acc[E][RF] = {};
  struct Step {
    Rows<E> x;
    Shared<RF * kP, kDyWaves> h;
    float back;
  };
  in_turn<Step, kAhead>(
      (c.n + kStep - 1) / kStep,
      [&](Step &v, int s) {
        const size_t step = c.step + s;
        size_t row[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) row[i] = static_cast<size_t>(max(tokens[s * kStep + 8 * q + i], 0)) * width;
        load_rows(v.x, dy, row, min(n0 + E * col, width - E));
        v.h.load(h.over + step * RF * kP * 64);
        if constexpr (DT == kF16) v.back = h.over_back[step * 16 * RF + min(static_cast<int>(threadIdx.x), 16 * RF - 1)];
      },
      [&](Step &v, int s) {
        const int i0 = c.i0 + s * kStep, n = min(c.n - s * kStep, kStep);
        uint16_t *lay = tile[wave];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int t = 8 * q + i;
          *reinterpret_cast<uint2 *>(lay + t * kCols + ((col >> 1) ^ (t & 7)) * 8 + 4 * (col & 1)) =
              make_uint2(v.x.w[i][0], v.x.w[i][1]);
        }
        v.h.lay(hs);
        if (DT == kF16 && threadIdx.x < 16 * RF) backs[threadIdx.x] = v.back;
        lds_barrier();
        // this wavefront's share of u
        float *mine = red[wave];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          float4_t d[RF] = {};
#pragma unroll
          for (int k = 0; k < kK; ++k) {
            const int t = 16 * f + col;
            const Oct a = load_oct_aligned(lay + t * kCols + ((4 * k + q) ^ (t & 7)) * 8);
#pragma unroll
            for (int g = 0; g < RF; ++g) d[g] = mfma<DT>(a, bv[k][g], d[g]);
          }
#pragma unroll
          for (int g = 0; g < RF; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) mine[(16 * f + 4 * q + i) * kStride + 16 * g + col] = d[g][i];
        }
        if (n < kStep) drop_rows(v.x, 8 * q, n);
        Oct x[E];
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = column(v.x, e);
#pragma unroll
        for (int g = 0; g < RF; ++g) {
          float4_t d[E] = {};
#pragma unroll
          for (int p = 0; p < kP; ++p) {
            const Oct w = hs[(g * kP + p) * 64 + lane];
#pragma unroll
            for (int e = 0; e < E; ++e) {
              if constexpr (DT == kF16) d[e] = mfma<DT>(x[e], w, d[e]);
              else acc[e][g] = mfma<DT>(x[e], w, acc[e][g]);
            }
          }
          if constexpr (DT == kF16) {
            const float back = backs[16 * g + col];
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[e][g][i] = fmaf(d[e][i], back, acc[e][g][i]);
          }
        }
        // the slice's share of u (what it reads, and hs, is written again behind the
        // next step's first barrier, or behind this one)
        lds_barrier();
        float *out = u_part + (static_cast<size_t>(blockIdx.x) * M + i0) * r;
        for (int i = threadIdx.x; i < kStep * 16 * RF; i += kDyThreads) {
          const int t = i / (16 * RF), j = i % (16 * RF);
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < kDyWaves; ++w) sum += red[w][t * kStride + j];
          if (t < n && j < r) out[t * r + j] = sum;
        }
      });
  const float sa = scales[c.a];
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int g = 0; g < RF; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = n0 + E * (4 * q + i), n = min(m, width - E) + e, j = 16 * g + col;
        if (n >= m && n < N && j < r)
          put(dB, part, c, static_cast<size_t>(N) * r, static_cast<size_t>(n) * r + j, acc[e][g][i], sa);
      }
}

// ------------------------------------------------------------------ x: dA and dx

// Workgroup (chunk, slice of 256 columns) as above; A's operands stay in registers, a
// step's operands of u go through LDS to the four wavefronts. Bound by HBM: 8192
// tokens, 4096 columns 44 us at rank 16 (201 MB with base, 4.6 TB/s), 58 at rank 64.
template <int DT, int RF>
__global__ void __launch_bounds__(kThreads, RF <= 4 ? 2 : 1) adapters_x_kernel(
    const uint16_t *__restrict__ x, int M, int K, int r, const uint16_t *__restrict__ A, int L,
    const int32_t *__restrict__ ids, const int32_t *__restrict__ offsets, const int32_t *__restrict__ perm, int rows,
    int chunks, int max_steps, Pieces u, const uint16_t *base, uint16_t *dx, float *__restrict__ dA,
    float *__restrict__ part) {
  constexpr int E = kE, kP = kPieces<DT>, kOps = kOperands<DT, RF>, kCols = 16 * E, kSlice = kCols * kWaves;
  __shared__ Oct over[RF * kP * 64], along[2 * kOps * 64];
  __shared__ __attribute__((aligned(16))) float backs[16 * RF];
  __shared__ __attribute__((aligned(16))) int tokens[kMostTokens];
  __shared__ int list[64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
  const int s0 = blockIdx.x * kSlice, s1 = min(K, s0 + kSlice);
  if (static_cast<int>(blockIdx.y) >= chunks + L)   // 64 tokens: those without an adapter
    return copy_others<kThreads>(ids, (blockIdx.y - chunks - L) * 64, M, L, base, dx, K, s0, s1, list);
  if (static_cast<int>(blockIdx.y) >= chunks) {
    int lo, hi;
    const int a = blockIdx.y - chunks;
    segment(offsets, a, M, lo, hi);
    // (no tokens: zeros, an equal share of the adapter's to every slice)
    const size_t all = static_cast<size_t>(r) * K / 4, from = all * blockIdx.x / gridDim.x;
    if (lo == hi)
      clear<kThreads>(dA + 4 * (all * a + from), 4 * (all * (blockIdx.x + 1) / gridDim.x - from));
    return;
  }
  const Chunk c = chunk_of(offsets, L, M, rows, kStep, max_steps, blockIdx.y);
  if (c.a < 0) return;
  stage_tokens(perm, c, kStep, M, tokens);
  // (K is a multiple of 128: a wavefront's columns are all there or none is; those of
  // none go along, for the barriers, on the last ones, and store nothing)
  const bool mine = s0 + wave * kCols < K;
  const int k0 = mine ? s0 + wave * kCols : K - kCols;
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
      load_rows(v, Aa, row, k0 + E * col);
      drop_rows(v, j, r);
#pragma unroll
      for (int e = 0; e < E; ++e) av[e][g] = column(v, e);
    }
  }
  float4_t acc[E][RF] = {};
  struct Step {
    Rows<E> x;
    Rows<E, 4> base[2];
    Shared<RF * kP, kWaves> over;
    Shared<2 * kOps, kWaves> along;
    float back;
    float4_t token_back[2];
  };
  // (a step ahead costs more registers than there are from rank 17 on: all launches of 4000
  // tokens of 96 adapters, rank 32, with it 80 us, without 70; 8192 tokens, rank 64, bf16, 347
  // and 260)
  constexpr int kAhead = RF >= 2 ? 0 : 1;
  in_turn<Step, kAhead>(
      (c.n + kStep - 1) / kStep,
      [&](Step &v, int s) {
        const size_t step = c.step + s;
        const int *at32 = tokens + s * kStep;
        size_t row[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) row[i] = static_cast<size_t>(max(at32[8 * q + i], 0)) * K;
        load_rows(v.x, x, row, k0 + E * col);
        if (base) {
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            size_t at[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) at[i] = static_cast<size_t>(max(at32[16 * f + 4 * q + i], 0)) * K;
            load_rows(v.base[f], base, at, k0 + E * col);
          }
        } else {
          v.base[0] = v.base[1] = Rows<E, 4>{};
        }
        v.over.load(u.over + step * RF * kP * 64);
        v.along.load(u.along + step * 2 * kOps * 64);
        if constexpr (DT == kF16) {
          v.back = u.over_back[step * 16 * RF + min(static_cast<int>(threadIdx.x), 16 * RF - 1)];
#pragma unroll
          for (int f = 0; f < 2; ++f)
            v.token_back[f] = *reinterpret_cast<const float4_t *>(u.along_back + step * kStep + 16 * f + 4 * q);
        }
      },
      [&](Step &v, int s) {
        const int n = min(c.n - s * kStep, kStep);
        lds_barrier();   // the step before has read its operands
        v.over.lay(over);
        v.along.lay(along);
        if (DT == kF16 && threadIdx.x < 16 * RF) backs[threadIdx.x] = v.back;
        lds_barrier();
        if (n < kStep) drop_rows(v.x, 8 * q, n);
        Oct xv[E];
#pragma unroll
        for (int e = 0; e < E; ++e) xv[e] = column(v.x, e);
#pragma unroll
        for (int g = 0; g < RF; ++g) {
          float4_t d[E] = {};
#pragma unroll
          for (int p = 0; p < kP; ++p) {
            const Oct w = over[(g * kP + p) * 64 + lane];
#pragma unroll
            for (int e = 0; e < E; ++e) {
              if constexpr (DT == kF16) d[e] = mfma<DT>(w, xv[e], d[e]);
              else acc[e][g] = mfma<DT>(w, xv[e], acc[e][g]);
            }
          }
          if constexpr (DT == kF16) {
            const float4_t back = *reinterpret_cast<const float4_t *>(backs + 16 * g + 4 * q);
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[e][g][i] = fmaf(d[e][i], back[i], acc[e][g][i]);
          }
        }
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          // D's rows are tokens: a lane holds columns k0 + E col .. of tokens 4 q .. + 3
          float4_t d[E] = {};
#pragma unroll
          for (int k = 0; k < kOps; ++k) {
            const Oct w = along[(f * kOps + k) * 64 + lane];
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] = mfma<DT>(w, beside(av[e], k, q), d[e]);
          }
          size_t at[4];
          bool live[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = 16 * f + 4 * q + i, to = tokens[s * kStep + t];
            live[i] = mine && t < n && to >= 0;
            at[i] = static_cast<size_t>(max(to, 0)) * K;
          }
          const float4_t back = DT == kF16 ? v.token_back[f] : float4_t{1.f, 1.f, 1.f, 1.f};
          add_rows<DT, E>(dx, at, live, k0 + E * col, 0, K, d, back, v.base[f]);
        }
      });
  if (!mine) return;
#pragma unroll
  for (int g = 0; g < RF; ++g)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = 16 * g + 4 * q + i;
      if (j >= r) continue;
      const size_t at = static_cast<size_t>(j) * K + k0 + E * col;
      const size_t size = static_cast<size_t>(r) * K;
      float *out = c.slot >= 0 ? part + static_cast<size_t>(c.slot) * size : dA + static_cast<size_t>(c.a) * size;
      *reinterpret_cast<float4_t *>(out + at) = float4_t{acc[0][g][i], acc[1][g][i], acc[2][g][i], acc[3][g][i]};
    }
}

// The chunks' sums of the adapters that have several, added up in order. Bound by
// reading them (16 chunks of 14336 x 16 values 7.4 us).
__global__ void __launch_bounds__(kThreads) adapters_sum_kernel(const float *__restrict__ part, size_t size, int M,
                                                                const float *__restrict__ scales,
                                                                const int32_t *__restrict__ offsets, int rows,
                                                                float *__restrict__ out) {
  const int a = blockIdx.y;
  int lo, hi;
  segment(offsets, a, M, lo, hi);
  if (hi - lo <= rows) return;
  const int each = cut_of(hi - lo, rows, kStep).each;
  const float sa = scales ? scales[a] : 1.f;
  for (size_t i = static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x; i < size;
       i += static_cast<size_t>(gridDim.x) * kThreads) {
    float s = 0.f;
#pragma unroll 8
    for (int at = lo; at < hi; at += each) s += part[static_cast<size_t>(slot_of(at, rows, hi - at <= each)) * size + i];
    out[static_cast<size_t>(a) * size + i] = s * sa;
  }
}

// ------------------------------------------------------------------ plan

constexpr size_t kAlign = 256;
size_t round_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

struct Plan {
  int rf;
  int steps;                    // at most
  int rows_y, chunks_y, rows_x, chunks_x;
  int slices_y, slices_x;
  size_t over, along, over_back, along_back, u_part, sums, pad, total;   // where in the workspace
};

// Tokens of a chunk: so many that the workgroups of all slices fill `slots` once, and
// one step at least (257 tokens, 2048 columns, rank 5: dy 11.4 and x 10.7 us with at
// least 128, 7.3 and 6.9 with 32; 2000 tokens on two adapters, 4096 columns, rank 64 all
// launches 79 and 74). Where tokens lie together by many adapters a larger least would
// have fewer sums to add up: 4000 tokens on 96, 2048 columns, rank 32 62 and 84.
int chunk_rows(int M, int slices, int slots) {
  const long rows = (static_cast<long>(M) * slices + slots - 1) / slots;
  return static_cast<int>(std::min<long>(std::max<long>((rows + kStep - 1) / kStep * kStep, 32), kMostTokens));
}

Plan plan_of(const AdapterArgs &g) {
  Plan p{};
  const int frags = (g.r + 15) / 16;
  p.rf = frags <= 1 ? 1 : frags <= 2 ? 2 : frags <= 4 ? 4 : 8;
  p.slices_y = (g.N + 16 * kE * dy_waves(p.rf) - 1) / (16 * kE * dy_waves(p.rf));
  p.slices_x = (g.K + 16 * kE * kWaves - 1) / (16 * kE * kWaves);
  const int some = std::min(g.L, g.M);
  p.steps = g.M / kStep + some;
  p.rows_y = chunk_rows(g.M, p.slices_y, p.rf == 1 ? 512 : 256);
  p.rows_x = chunk_rows(g.M, p.slices_x, 512);
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
  p.along = take(static_cast<size_t>(p.steps) * 2 * operands_of(g.dtype, p.rf) * 64 * sizeof(Oct));
  p.over_back = take(static_cast<size_t>(p.steps) * 16 * p.rf * 4);
  p.along_back = take(static_cast<size_t>(p.steps) * kStep * 4);
  p.u_part = take(static_cast<size_t>(p.slices_y) * g.M * g.r * 4);
  const size_t sums_y = g.M > p.rows_y ? 2 * (static_cast<size_t>(g.M) / (p.rows_y / 2) + 1) * g.N * g.r * 4 : 0;
  const size_t sums_x = g.M > p.rows_x ? 2 * (static_cast<size_t>(g.M) / (p.rows_x / 2) + 1) * g.K * g.r * 4 : 0;
  p.sums = take(std::max(sums_y, sums_x));   // dB's are done with when dA's begin
  p.pad = take(g.N < kNarrow ? static_cast<size_t>(g.M) * kNarrow * 2 : 0);
  p.total = at;
  return p;
}

template <int DT, int RF>
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
    hipLaunchKernelGGL((adapters_pieces_kernel<DT, RF, true>), dim3(p.steps), dim3(kPieceThreads), 0, s, g.h, 1, g.M, g.r, g.scales,
                       g.L, g.offsets, g.perm, q);
  const uint16_t *dy = static_cast<const uint16_t *>(g.dy);
  if (g.M > 0 && g.N < kNarrow) {
    uint16_t *pad = reinterpret_cast<uint16_t *>(ws + p.pad);
    hipLaunchKernelGGL(adapters_pad_kernel<kThreads>, dim3((g.M * kNarrow + kThreads - 1) / kThreads), block, 0, s, dy,
                       g.M, g.N, pad);
    dy = pad;
  }
  hipLaunchKernelGGL((adapters_dy_kernel<DT, RF>), dim3(p.slices_y, p.chunks_y + g.L), dim3(64 * dy_waves(RF)), 0, s, dy,
                     std::max(g.N, kNarrow), g.M, g.N, g.r, b, g.scales, g.L, g.offsets, g.perm, p.rows_y,
                     p.chunks_y, p.steps, q, u_part, g.d_b, sums);
  if (g.M > p.rows_y) sum(static_cast<size_t>(g.N) * g.r, g.scales, p.rows_y, g.d_b);
  if (p.steps > 0)
    hipLaunchKernelGGL((adapters_pieces_kernel<DT, RF, false>), dim3(p.steps), dim3(kPieceThreads), 0, s, u_part, p.slices_y, g.M, g.r,
                       g.scales, g.L, g.offsets, g.perm, q);
  const int others = base == dx ? 0 : (g.M + 63) / 64;
  hipLaunchKernelGGL((adapters_x_kernel<DT, RF>), dim3(p.slices_x, p.chunks_x + g.L + others), block, 0, s,
                     static_cast<const uint16_t *>(g.x), g.M, g.K, g.r, a, g.L, g.ids, g.offsets, g.perm, p.rows_x,
                     p.chunks_x, p.steps, q, base, dx, g.d_a, sums);
  if (g.M > p.rows_x) sum(static_cast<size_t>(g.K) * g.r, nullptr, p.rows_x, g.d_a);
}

template <int DT>
void backward_ranks(const AdapterArgs &g, const Plan &p, hipStream_t s) {
  if (p.rf == 1) backward_go<DT, 1>(g, p, s);
  else if (p.rf == 2) backward_go<DT, 2>(g, p, s);
  else if (p.rf == 4) backward_go<DT, 4>(g, p, s);
  else backward_go<DT, 8>(g, p, s);
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
