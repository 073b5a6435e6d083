// Products of MXFP4 tensors: y[i][n] = sum_k a[i][k] b[n][k], dense and grouped
// over experts, on v_mfma_scale_f32_32x32x64_f8f6f4 (both operands fp4, the
// E8M0 scales applied inside the instruction, fp32 accumulation).
//
// Operand layout of the instruction: lane (r, h), r = lane & 31, h = lane >> 5,
// holds the 32 values of row r, block h of the 64-long step (16 bytes) and that
// block's scale byte; result register i of lane (c, h) is row
// 8 (i / 4) + 4 h + i % 4, column c.
#include "device.h"
#include "gemm_common.h"
#include "kernels.h"
#include "mxfp4.h"
#include "mx_tiles.h"

#include <algorithm>

namespace lbq {

namespace {

using namespace mxfp4;

typedef float v16f_t __attribute__((ext_vector_type(16)));

struct GemmArgs {
  const uint8_t *a_codes;      // [a_rows][K / 2]
  const uint32_t *a_scales;    // [K / 128][a_rows]
  const uint8_t *b_codes;      // [b_rows][K / 2], b_rows = E N
  const uint32_t *b_scales;    // [K / 128][b_rows]
  void *y;                     // [M or T][N]
  int a_rows, b_rows, M, N, K;
  // grouped: list rows by expert; perm[i] / top_k (or i) is the activation row
  const int32_t *offsets, *perm;
  int E, top_k;
  int tiles_m, tiles_n;
};

// A workgroup of GM x GN waves; a wave owns MB x NB blocks of 32 tokens by 32
// weight rows. The weight is the instruction's first operand, so a lane's four
// consecutive result registers are four neighbouring outputs of one token.
//
// Stages of one 128-group of K (64 bytes and a scale word a row) go global -> LDS
// by asynchronous copies into a ring of RING buffers. In stage s the copies of
// stages s + 2 .. s + RING - 1 are in flight and the operands of the next
// 64-long step are read from LDS while one step is multiplied, across the stage's
// border too: stage s starts when s + 1 has landed. One barrier per stage. Vector
// v (16 bytes) of row r lies in slot v ^ ((r >> 2) & 3) of the row: the sixteen
// rows that a quarter of an operand read touches fall in sixteen distinct 16-byte
// bank groups. Stages of two groups (128 bytes a row) leave fewer workgroups per
// compute unit and measured slower (256 experts, 2048 tokens: 193 -> 210 us).
template <int MB, int NB, int GM, int GN>
struct Tile {
  static constexpr int kThreads = 64 * GM * GN, kVecs = 4;   // 16-byte vectors of a row's stage
  static constexpr int kM = 32 * MB * GM, kN = 32 * NB * GN;
  static constexpr int kCopiesA = kM * kVecs / kThreads, kCopiesB = kN * kVecs / kThreads;
  static_assert(kCopiesA * kThreads == kM * kVecs && kCopiesB * kThreads == kN * kVecs, "whole copies");
  // scale words: where a tile has fewer rows than threads, the waves without rows
  // copy one word (so that every wave has the same number of copies in flight)
  static constexpr int kScalesA = kM < kThreads ? 1 : kM / kThreads, kScalesB = kN < kThreads ? 1 : kN / kThreads;
  static_assert(kM % 64 == 0 && kN % 64 == 0, "a wave copies 64 scale words");
  static constexpr int kLoads = kCopiesA + kCopiesB + kScalesA + kScalesB;   // per wave and stage
};

// One stage's buffer, an object of its own: the compiler tells reads of one
// from copies in flight into another.
template <class Tl>
struct Stage {
  uint4 a[Tl::kM * Tl::kVecs], b[Tl::kN * Tl::kVecs];
  uint32_t sa[Tl::kM], sb[Tl::kN], idle[64];
};

// Tile number -> (row tile, column tile): `group` row tiles down each column
// before the next.
__device__ __forceinline__ void place_tile(int id, int tm, int tn, int group, int &m, int &n) {
  const int width = group * tn, g = id / width, first = g * group;
  const int rows = min(tm - first, group), in = id - g * width;
  m = first + in % rows;
  n = in / rows;
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return from_f32<DT>(a) | (static_cast<uint32_t>(from_f32<DT>(b)) << 16);
}

// One 32 x 32 result block: token row m (the lane's), outputs n0 .. n0 + 31.
// VEC: N is a multiple of 8, so eight neighbouring outputs (four in fp32) are
// one aligned 16-byte store. The halves of a token's outputs sit in lanes
// (m, 0) and (m, 1); a lane swap gives each eight neighbours.
template <int DT, bool VEC>
__device__ __forceinline__ void store_block(void *y, size_t row, bool ok, int n0, int N, int h, const v16f_t &acc) {
  using T = typename Elem<DT>::type;
  if constexpr (VEC && DT != kF32) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      uint32_t a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[i] = pack2<DT>(acc[8 * q + 2 * i], acc[8 * q + 2 * i + 1]);
        b[i] = pack2<DT>(acc[8 * q + 4 + 2 * i], acc[8 * q + 4 + 2 * i + 1]);
        const auto sw = __builtin_amdgcn_permlane32_swap(a[i], b[i], false, false);
        a[i] = sw[0];
        b[i] = sw[1];
      }
      const int n = n0 + 16 * q + 8 * h;
      if (ok && n < N) *reinterpret_cast<uint4 *>(static_cast<T *>(y) + row * N + n) = make_uint4(a[0], a[1], b[0], b[1]);
    }
  } else if constexpr (VEC) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int n = n0 + 8 * q + 4 * h;
      if (ok && n < N)
        *reinterpret_cast<float4_t *>(static_cast<T *>(y) + row * N + n) =
            float4_t{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
    }
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int n = n0 + 8 * (k / 4) + 4 * h + k % 4;
      if (ok && n < N) static_cast<T *>(y)[row * N + n] = from_f32<DT>(acc[k]);
    }
  }
}

template <int MB, int NB, int GM, int GN, int RING, int DT, bool GROUPED>
__global__ void __launch_bounds__(64 * GM *GN, 1) mx_tile_kernel(GemmArgs g) {
  using Tl = Tile<MB, NB, GM, GN>;
  using Buffer = Stage<Tl>;
  constexpr int TH = Tl::kThreads, CA = Tl::kCopiesA, CB = Tl::kCopiesB;
  static_assert(RING == 3 || RING == 4, "ring");
  __shared__ __attribute__((aligned(16))) Buffer q0, q1, q2, q3;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;
  int tile_m, tile_n, i0, n_rows, e = 0;
  if constexpr (GROUPED) {
    const GroupTiles tiles(g.offsets, g.E, g.M, Tl::kM);
    const int tm = tiles.total(), id = xcd_order(blockIdx.x, tm * g.tiles_n);
    if (id < 0) return;
    place_tile(id, tm, g.tiles_n, 4, tile_m, tile_n);
    const GroupTile t = tiles.find(tile_m);
    i0 = t.i0;
    n_rows = t.n;
    e = t.e;
  } else {
    place_tile(xcd_order(blockIdx.x, g.tiles_m * g.tiles_n), g.tiles_m, g.tiles_n, 4, tile_m, tile_n);
    i0 = tile_m * Tl::kM;
    n_rows = g.M - i0;
  }
  const int col0 = tile_n * Tl::kN;
  // K slice blockIdx.y: S stages from stage `first` on
  const int all = g.K / kGroup, first = static_cast<int>(static_cast<long>(all) * blockIdx.y / gridDim.y);
  const int S = static_cast<int>(static_cast<long>(all) * (blockIdx.y + 1) / gridDim.y) - first;
  // activation row of list row i0 + i (rows past the end repeat the last one;
  // their results are not stored)
  auto act_row = [&](int i) {
    int ia = i0 + min(i, n_rows - 1);
    if constexpr (GROUPED)
      if (g.perm) ia = g.perm[ia] / g.top_k;
    return static_cast<size_t>(min(max(ia, 0), g.a_rows - 1));
  };
  auto weight_row = [&](int n) { return static_cast<size_t>(e) * g.N + min(col0 + n, g.N - 1); };
  constexpr int kVecs = Tl::kVecs;
  const int vec = (tid % kVecs) ^ ((tid >> 4) % kVecs);
  const uint8_t *pa[CA], *pb[CB];
#pragma unroll
  for (int it = 0; it < CA; ++it)
    pa[it] = g.a_codes + act_row((it * TH + tid) / kVecs) * (g.K / 2) + 64 * first + 16 * vec;
#pragma unroll
  for (int it = 0; it < CB; ++it)
    pb[it] = g.b_codes + weight_row((it * TH + tid) / kVecs) * (g.K / 2) + 64 * first + 16 * vec;
  const uint32_t *psa[Tl::kScalesA], *psb[Tl::kScalesB];
#pragma unroll
  for (int it = 0; it < Tl::kScalesA; ++it)
    psa[it] = g.a_scales + static_cast<size_t>(first) * g.a_rows + act_row(it * TH + tid < Tl::kM ? it * TH + tid : 0);
#pragma unroll
  for (int it = 0; it < Tl::kScalesB; ++it)
    psb[it] = g.b_scales + static_cast<size_t>(first) * g.b_rows + weight_row(it * TH + tid < Tl::kN ? it * TH + tid : 0);

  // copies of the next stage in line; past the last one it repeats, so that
  // every stage has the same number of copies in flight (never multiplied)
  int ahead = 0;
  auto issue = [&](Buffer &q) {
#pragma unroll
    for (int it = 0; it < CA; ++it) copy16_to_lds(pa[it], q.a + it * TH + wave * 64);
#pragma unroll
    for (int it = 0; it < CB; ++it) copy16_to_lds(pb[it], q.b + it * TH + wave * 64);
#pragma unroll
    for (int it = 0; it < Tl::kScalesA; ++it)
      copy4_to_lds(psa[it], it * TH + wave * 64 < Tl::kM ? q.sa + it * TH + wave * 64 : q.idle);
#pragma unroll
    for (int it = 0; it < Tl::kScalesB; ++it)
      copy4_to_lds(psb[it], it * TH + wave * 64 < Tl::kN ? q.sb + it * TH + wave * 64 : q.idle);
    const bool more = ++ahead < S;
    const int by = more ? 64 : 0;
    const size_t da = more ? g.a_rows : 0, db = more ? g.b_rows : 0;
#pragma unroll
    for (int it = 0; it < CA; ++it) pa[it] += by;
#pragma unroll
    for (int it = 0; it < CB; ++it) pb[it] += by;
#pragma unroll
    for (int it = 0; it < Tl::kScalesA; ++it) psa[it] += da;
#pragma unroll
    for (int it = 0; it < Tl::kScalesB; ++it) psb[it] += db;
  };

  const int wm = (wave / GN) * 32 * MB, wn = (wave % GN) * 32 * NB;
  const int key = (r >> 2) % kVecs;
  v16f_t acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[i][j][k] = 0.f;

  struct Step {
    v8i_t a[MB], b[NB];
  };
  struct Scales {   // words of one group: bytes 0 and 2 are this lane's blocks of its two steps
    uint32_t a[MB], b[NB];
  };
  auto read = [&](Step &f, const Buffer &q, int s) {
    const int at = (2 * s + h) ^ key;
#pragma unroll
    for (int j = 0; j < NB; ++j) f.b[j] = operand(q.b[(wn + 32 * j + r) * kVecs + at]);
#pragma unroll
    for (int i = 0; i < MB; ++i) f.a[i] = operand(q.a[(wm + 32 * i + r) * kVecs + at]);
  };
  auto read_scales = [&](Scales &v, const Buffer &q) {
#pragma unroll
    for (int i = 0; i < MB; ++i) v.a[i] = q.sa[wm + 32 * i + r] >> (8 * h);
#pragma unroll
    for (int j = 0; j < NB; ++j) v.b[j] = q.sb[wn + 32 * j + r] >> (8 * h);
  };
#define LBQ_MX_STEP(F, SEL, V)                                                                                  \
  do {                                                                                                          \
    _Pragma("unroll") for (int i = 0; i < MB; ++i) _Pragma("unroll") for (int j = 0; j < NB; ++j) acc[i][j] =   \
        __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(F.b[j], F.a[i], acc[i][j], 4, 4, SEL,                   \
                                                        static_cast<int>(V.b[j]), SEL, static_cast<int>(V.a[i])); \
  } while (0)

  Step f0, f1;
  Scales v0, v1;
  // After a wait for its own copies: every wave's have landed, and every wave is
  // done with its reads so far.
  auto meet = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  // Stage in cur, its first step's operands in f0, its first scales in v0; free
  // takes the copies. The order of the instructions: LDS reads (a step's, while
  // the step before it is multiplied), then copies, one by one between products,
  // so that neither holds up the matrix cores (8192 x 4096 x 14336: 261 -> 243 us
  // against the compiler's own order).
  auto stage = [&](const Buffer &cur, const Buffer &next, Buffer &free) {
    wait_vm_lds<(RING - 3) * Tl::kLoads>();   // the stage after this one
    meet();
    issue(free);
    read(f1, cur, 1);
    LBQ_MX_STEP(f0, 0, v0);
    v1 = v0;
    read(f0, next, 0);
    read_scales(v0, next);
    LBQ_MX_STEP(f1, 2, v1);
    constexpr int kP = MB * NB, kR = MB + NB;
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (i < kR) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if (i >= kR) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
    }
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (i < kR) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      if (i >= kR) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
    }
  };
  issue(q0);
  issue(q1);
  if constexpr (RING == 4) issue(q2);
  wait_vm_lds<(RING - 2) * Tl::kLoads>();
  meet();
  read(f0, q0, 0);
  read_scales(v0, q0);
  // whole rounds of the ring, then what is left of one (no exits inside the
  // loop: the accumulators keep their registers)
  const int rest = S % RING;
  for (int n = S / RING; n > 0; --n) {
    if constexpr (RING == 4) {
      stage(q0, q1, q3);
      stage(q1, q2, q0);
      stage(q2, q3, q1);
      stage(q3, q0, q2);
    } else {
      stage(q0, q1, q2);
      stage(q1, q2, q0);
      stage(q2, q0, q1);
    }
  }
  if (rest > 0) {
    if constexpr (RING == 4) stage(q0, q1, q3);
    else stage(q0, q1, q2);
  }
  if (rest > 1) {
    if constexpr (RING == 4) stage(q1, q2, q0);
    else stage(q1, q2, q0);
  }
  if constexpr (RING == 4)
    if (rest > 2) stage(q2, q3, q1);
#undef LBQ_MX_STEP
  wait_vm_lds<0>();   // no copy into LDS outlives the workgroup
  const bool vecs = g.N % 8 == 0;
  // slices write partial results one behind the other
  void *y = g.y;
  if constexpr (DT == kF32) y = static_cast<float *>(y) + static_cast<size_t>(blockIdx.y) * g.M * g.N;
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int row = wm + 32 * i + r;
    const size_t at = static_cast<size_t>(i0) + row;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int n0 = col0 + wn + 32 * j;
      if (vecs) store_block<DT, true>(y, at, row < n_rows, n0, g.N, h, acc[i][j]);
      else store_block<DT, false>(y, at, row < n_rows, n0, g.N, h, acc[i][j]);
    }
  }
}

// Sum of S partial results in slice order, rounded once.
__global__ void __launch_bounds__(256) mx_sum_kernel(const float *__restrict__ part, int S, long n, int dtype,
                                                     void *__restrict__ y) {
  for (long i = static_cast<long>(blockIdx.x) * 256 + threadIdx.x; i < n; i += 256l * gridDim.x) {
    float v = part[i];
    for (int k = 1; k < S; ++k) v += part[k * n + i];
    if (dtype == kF16) static_cast<uint16_t *>(y)[i] = from_f32<kF16>(v);
    else if (dtype == kBF16) static_cast<uint16_t *>(y)[i] = from_f32<kBF16>(v);
    else static_cast<float *>(y)[i] = v;
  }
}

template <int MB, int NB, int GM, int GN, int RING>
hipError_t launch_tiles(GemmArgs g, int dtype, int slices, hipStream_t s) {
  using Tl = Tile<MB, NB, GM, GN>;
  // grouped: every expert may end in a ragged tile
  const long tm = (static_cast<long>(g.M) + Tl::kM - 1) / Tl::kM + (g.E > 0 ? std::min(g.E, g.M) : 0);
  const long tn = (static_cast<long>(g.N) + Tl::kN - 1) / Tl::kN;
  if (tm * tn >= (1l << 31)) return hipErrorInvalidValue;
  g.tiles_m = static_cast<int>(tm);
  g.tiles_n = static_cast<int>(tn);
  const dim3 grid(static_cast<unsigned>(tm * tn), static_cast<unsigned>(slices)), block(Tl::kThreads);
#define LBQ_MX_GO(DT)                                                                                       \
  if (g.E > 0) hipLaunchKernelGGL((mx_tile_kernel<MB, NB, GM, GN, RING, DT, true>), grid, block, 0, s, g);        \
  else hipLaunchKernelGGL((mx_tile_kernel<MB, NB, GM, GN, RING, DT, false>), grid, block, 0, s, g)
  if (dtype == kF16) {
    LBQ_MX_GO(kF16);
  } else if (dtype == kBF16) {
    LBQ_MX_GO(kBF16);
  } else {
    LBQ_MX_GO(kF32);
  }
#undef LBQ_MX_GO
  return hipGetLastError();
}

// Which tile, and how many slices of K.
//
// Dense: a workgroup per compute unit takes, per 4096 of K, about 41 us on 256 x
// 256, 13.6 on 128 x 128 and 8.7 on 64 x 128 (4096^3 and 512 x 4096^2); the
// smallest sum of rounds wins. Fewer tiles of the smallest kind than half the
// compute units: K in slices of at least 1024.
//
// Grouped, by the average expert's rows: 64 x 256 to 96 rows, where the experts'
// weights are what has to move (256 experts of 2048 x 2048, 64 rows: 181 us;
// 128 x 128 193, 256 x 256 226), 128 x 128 below 512 (8 experts of 4096 x 4096,
// 128 rows: 31 us; 36 and 37), else 256 x 256 (28672 x 4096, 2048 rows: 1.39 ms;
// 128 x 128 1.71).
struct Plan {
  int bm, bn, slices;
};
Plan plan_tiles(const MxGemm &p) {
  if (p.E > 0) {
    const int avg = p.M / p.E;
    if (avg <= 96) return {64, p.N <= 128 ? 128 : 256, 1};
    return avg < 512 ? Plan{128, 128, 1} : Plan{256, 256, 1};
  }
  auto tiles = [&](int bm, int bn) {
    return ((static_cast<long>(p.M) + bm - 1) / bm) * ((static_cast<long>(p.N) + bn - 1) / bn);
  };
  auto rounds = [&](int bm, int bn) { return static_cast<double>((tiles(bm, bn) + 255) / 256); };
  const double big = 41 * rounds(256, 256), mid = 13.6 * rounds(128, 128), small = 8.7 * rounds(64, 128);
  if (big <= mid && big <= small) return {256, 256, 1};
  if (mid <= small) return {128, 128, 1};
  Plan r{64, 128, 1};
  while (r.slices < 8 && tiles(64, 128) * r.slices * 2 <= 256 && p.K / (r.slices * 2) >= 1024) r.slices *= 2;
  return r;
}

}  // namespace

size_t mx_gemm_scratch_bytes(const MxGemm &p) {
  const Plan r = plan_tiles(p);
  return r.slices > 1 ? static_cast<size_t>(r.slices) * p.M * p.N * 4 : 0;
}

hipError_t launch_mx_gemm(const MxGemm &p, hipStream_t s) {
  const Plan r = plan_tiles(p);
  GemmArgs g{};
  g.a_codes = static_cast<const uint8_t *>(p.a_codes);
  g.a_scales = static_cast<const uint32_t *>(p.a_scales);
  g.b_codes = static_cast<const uint8_t *>(p.b_codes);
  g.b_scales = static_cast<const uint32_t *>(p.b_scales);
  g.y = r.slices > 1 ? p.scratch : p.y;
  g.a_rows = p.a_rows;
  g.b_rows = p.E > 0 ? p.E * p.N : p.N;
  g.M = p.M;
  g.N = p.N;
  g.K = p.K;
  g.offsets = p.offsets;
  g.perm = p.perm;
  g.E = p.E;
  g.top_k = p.top_k;
  const int dtype = r.slices > 1 ? kF32 : p.dtype;
  hipError_t e;
  if (r.bm == 256) e = launch_tiles<4, 4, 2, 2, 4>(g, dtype, r.slices, s);
  else if (r.bm == 128) e = launch_tiles<2, 2, 2, 2, 3>(g, dtype, r.slices, s);
  else if (r.bn == 256) e = launch_tiles<2, 2, 1, 4, 3>(g, dtype, r.slices, s);
  else e = launch_tiles<1, 2, 2, 2, 4>(g, dtype, r.slices, s);
  if (e != hipSuccess || r.slices == 1) return e;
  const long n = static_cast<long>(p.M) * p.N;
  hipLaunchKernelGGL(mx_sum_kernel, dim3(static_cast<unsigned>(std::min<long>((n + 255) / 256, 2048))), dim3(256), 0, s,
                     static_cast<const float *>(p.scratch), r.slices, n, p.dtype, p.y);
  return hipGetLastError();
}

}  // namespace lbq
