// Products of MXFP4 tensors: y[i][n] = sum_k a[i][k] b[n][k], dense and grouped
// over experts, on v_mfma_scale_f32_32x32x64_f8f6f4 (both operands fp4, the
// E8M0 scales applied inside the instruction, fp32 accumulation).
//
// Operand layout of the instruction: lane (r, h), r = lane & 31, h = lane >> 5,
// holds the 32 values of row r, block h of the 64-long step (16 bytes) and that
// block's scale byte; result register i of lane (c, h) is row
// 8 (i / 4) + 4 h + i % 4, column c.
//
// Bound: with many rows the matrix cores at the clock that the power limit leaves
// (6.3 PFLOP/s without any loads, on random codes), the copies into LDS beside
// them, and the results' way out after each tile. 8192 tokens 4096 -> 14336 279
// us, 3.4 PFLOP/s; 14336 -> 4096 255 us, 3.8; matrix cores 0.40 and 0.43 busy. With
// few rows per expert, HBM and the start and end of each tile (256 experts of
// 2048 x 2048, 64 rows each: 654 MB fetched in 169 us, 3.9 TB/s).
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
// Stages of two 128-groups of K (128 bytes and two scale words a row) go global
// -> LDS by asynchronous copies into two buffers in turn. A copy of 64 lanes
// takes eight rows of 128 bytes: whole cache lines, for which the copies reach
// 50 to 56 bytes per cycle and compute unit; of 64-byte pieces only 28 to 30, too
// few for the matrix cores (256 x 256 tiles take 34 KB per 1024 cycles of
// products). The operands of the next 64-long step are read from LDS while one
// step is multiplied, across the stage's border too, with one barrier per stage:
// before a stage's last step all its operands are in registers and the next
// stage has landed, so the barrier frees this stage's buffer for the copies after
// next and opens the next one's. Vector v (16 bytes) of row r lies in slot
// v ^ ((r >> 1) & 7) of the row: the sixteen rows that a quarter of an operand
// read touches fall in sixteen distinct 16-byte bank groups.
template <int MB, int NB, int GM, int GN>
struct Tile {
  static constexpr int kThreads = 64 * GM * GN, kVecs = 8;   // 16-byte vectors of a row's stage
  static constexpr int kM = 32 * MB * GM, kN = 32 * NB * GN;
  static constexpr int kCopiesA = kM * kVecs / kThreads, kCopiesB = kN * kVecs / kThreads;
  static_assert(kCopiesA * kThreads == kM * kVecs && kCopiesB * kThreads == kN * kVecs, "whole copies");
  // scale words: where a tile has fewer rows than threads, the waves without rows
  // copy one word (cheaper than a branch around the copy)
  static constexpr int kScalesA = kM < kThreads ? 1 : kM / kThreads, kScalesB = kN < kThreads ? 1 : kN / kThreads;
  static_assert(kM % 64 == 0 && kN % 64 == 0, "a wave copies 64 scale words");
};

// One stage's buffer, an object of its own: the compiler tells reads of one
// from copies in flight into another.
template <class Tl>
struct Stage {
  uint4 a[Tl::kM * Tl::kVecs], b[Tl::kN * Tl::kVecs];
  uint32_t sa[2][Tl::kM], sb[2][Tl::kN], idle[64];   // idle: for copies without a row
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

// One 32 x 32 result block into LDS: the lane's token is a row at `at`, its
// outputs as they lie in y. The halves of a token's eight neighbouring 16-bit
// outputs sit in lanes (m, 0) and (m, 1); a lane swap gives each eight.
template <int DT>
__device__ __forceinline__ void place_block(uint8_t *at, int h, const v16f_t &acc) {
  if constexpr (DT == kF32) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<float4_t *>(at + 4 * (8 * q + 4 * h)) =
          float4_t{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
  } else {
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
      *reinterpret_cast<uint4 *>(at + 2 * (16 * q + 8 * h)) = make_uint4(a[0], a[1], b[0], b[1]);
    }
  }
}

template <int MB, int NB, int GM, int GN, int DT, bool GROUPED>
__global__ void __launch_bounds__(64 * GM *GN, 1) mx_tile_kernel(GemmArgs g) {
  using Tl = Tile<MB, NB, GM, GN>;
  using Buffer = Stage<Tl>;
  constexpr int TH = Tl::kThreads, CA = Tl::kCopiesA, CB = Tl::kCopiesB;
  __shared__ __attribute__((aligned(16))) Buffer q0, q1;
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
  // K slice blockIdx.y: S stages from stage `first` on. An odd number of groups
  // leaves the last stage of the last slice half full.
  const int all = g.K / kGroup, pairs = (all + 1) / 2;
  const int first = static_cast<int>(static_cast<long>(pairs) * blockIdx.y / gridDim.y);
  const int S = static_cast<int>(static_cast<long>(pairs) * (blockIdx.y + 1) / gridDim.y) - first;
  const bool half_last = 2 * (first + S) > all;
  // Activation row of list row i0 + i and weight row col0 + n, from the row the
  // tile's base pointers stand at (rows past the end repeat the last one; their
  // results are not stored). Offsets from there are 32-bit: a tile's rows, or
  // with perm all of A's.
  const int a_base = GROUPED ? 0 : i0;
  auto act_row = [&](int i) {
    int ia = i0 + min(i, n_rows - 1);
    if constexpr (GROUPED)
      if (g.perm) ia = g.perm[ia] / g.top_k;
    return static_cast<uint32_t>(min(max(ia, 0), g.a_rows - 1) - a_base);
  };
  auto weight_row = [&](int n) { return static_cast<uint32_t>(min(n, g.N - 1 - col0)); };
  const size_t b_base = static_cast<size_t>(e) * g.N + col0;
  constexpr int kVecs = Tl::kVecs;
  const uint32_t row_bytes = g.K / 2;
  const int vec = (tid % kVecs) ^ ((tid >> 4) % kVecs);
  uint32_t oa[CA], ob[CB], osa[Tl::kScalesA], osb[Tl::kScalesB];
#pragma unroll
  for (int it = 0; it < CA; ++it) oa[it] = act_row((it * TH + tid) / kVecs) * row_bytes + 16 * vec;
#pragma unroll
  for (int it = 0; it < CB; ++it) ob[it] = weight_row((it * TH + tid) / kVecs) * row_bytes + 16 * vec;
#pragma unroll
  for (int it = 0; it < Tl::kScalesA; ++it) osa[it] = act_row(it * TH + tid < Tl::kM ? it * TH + tid : 0);
#pragma unroll
  for (int it = 0; it < Tl::kScalesB; ++it) osb[it] = weight_row(it * TH + tid < Tl::kN ? it * TH + tid : 0);
  // where the next stage in line begins
  const uint8_t *pa = g.a_codes + static_cast<size_t>(a_base) * row_bytes + 128 * static_cast<size_t>(first);
  const uint8_t *pb = g.b_codes + b_base * row_bytes + 128 * static_cast<size_t>(first);
  const uint32_t *psa = g.a_scales + a_base + static_cast<size_t>(2 * first) * g.a_rows;
  const uint32_t *psb = g.b_scales + b_base + static_cast<size_t>(2 * first) * g.b_rows;

  // Copies of the next stage in line; past the last one it repeats (never
  // multiplied). A half-full stage repeats its first half. No branches: a stage's
  // products and copies stay one block for the scheduler.
  int ahead = 0;
  auto issue = [&](Buffer &q) {
    const bool half = half_last && ahead >= S - 1;
    const uint32_t back = half && vec >= 4 ? 64 : 0;
    const size_t second_a = half ? 0 : g.a_rows, second_b = half ? 0 : g.b_rows;
#pragma unroll
    for (int it = 0; it < CA; ++it) copy16_to_lds(pa + (oa[it] - back), q.a + it * TH + wave * 64);
#pragma unroll
    for (int it = 0; it < CB; ++it) copy16_to_lds(pb + (ob[it] - back), q.b + it * TH + wave * 64);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int it = 0; it < Tl::kScalesA; ++it)
        copy4_to_lds(psa + (u ? second_a : 0) + osa[it],
                     it * TH + wave * 64 < Tl::kM ? q.sa[u] + it * TH + wave * 64 : q.idle);
#pragma unroll
      for (int it = 0; it < Tl::kScalesB; ++it)
        copy4_to_lds(psb + (u ? second_b : 0) + osb[it],
                     it * TH + wave * 64 < Tl::kN ? q.sb[u] + it * TH + wave * 64 : q.idle);
    }
    const bool more = ++ahead < S;
    pa += more ? 128 : 0;
    pb += more ? 128 : 0;
    psa += more ? 2 * static_cast<size_t>(g.a_rows) : 0;
    psb += more ? 2 * static_cast<size_t>(g.b_rows) : 0;
  };

  const int wm = (wave / GN) * 32 * MB, wn = (wave % GN) * 32 * NB;
  const int key = (r >> 1) % kVecs;
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
  auto read_scales = [&](Scales &v, const Buffer &q, int u) {
#pragma unroll
    for (int i = 0; i < MB; ++i) v.a[i] = q.sa[u][wm + 32 * i + r] >> (8 * h);
#pragma unroll
    for (int j = 0; j < NB; ++j) v.b[j] = q.sb[u][wn + 32 * j + r] >> (8 * h);
  };
#define LBQ_MX_STEP(F, SEL, V)                                                                                  \
  do {                                                                                                          \
    _Pragma("unroll") for (int i = 0; i < MB; ++i) _Pragma("unroll") for (int j = 0; j < NB; ++j) acc[i][j] =   \
        __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(F.b[j], F.a[i], acc[i][j], 4, 4, SEL,                   \
                                                        static_cast<int>(V.b[j]), SEL, static_cast<int>(V.a[i])); \
  } while (0)

  Step f0, f1;
  Scales v0, v1;
  // Every copy and LDS read of this wave is done; past the barrier every wave's.
  auto meet = [&]() {
    wait_vm_lds<0>();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  // Stage in cur, its first step's operands in f0, its first scales in v0, the
  // next stage on its way into next. Between the products go, one by one, the LDS
  // reads of the step after (and in the last step the copies), so that neither
  // holds up the matrix cores.
  constexpr int kP = MB * NB, kR = MB + NB;
  auto stage = [&](Buffer &cur, const Buffer &next) {
    read(f1, cur, 1);
    LBQ_MX_STEP(f0, 0, v0);
    read(f0, cur, 2);
    read_scales(v1, cur, 1);
    LBQ_MX_STEP(f1, 2, v0);
    read(f1, cur, 3);
    LBQ_MX_STEP(f0, 0, v1);
#pragma unroll
    for (int u = 0; u < 3; ++u)
#pragma unroll
      for (int i = 0; i < kP; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (i < kR) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        if (u == 1 && i < kR) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // the scales
      }
    meet();
    issue(cur);
    read(f0, next, 0);
    read_scales(v0, next, 0);
    LBQ_MX_STEP(f1, 2, v1);
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x010, 2, 0);
      if (i < kR) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    }
  };
  issue(q0);
  meet();
  issue(q1);
  read(f0, q0, 0);
  read_scales(v0, q0, 0);
  // whole stages by twos, then what is left (no exits inside the loop: the
  // accumulators keep their registers)
  const int full = S - (half_last ? 1 : 0);
  for (int n = full / 2; n > 0; --n) {
    stage(q0, q1);
    stage(q1, q0);
  }
  const bool odd = full & 1;
  if (odd) stage(q0, q1);
  if (half_last) {
    read(f1, odd ? q1 : q0, 1);
    LBQ_MX_STEP(f0, 0, v0);
    LBQ_MX_STEP(f1, 2, v0);
  }
#undef LBQ_MX_STEP
  meet();   // no copy is under way any more, and no operand is read
  // slices write partial results one behind the other
  using T = typename Elem<DT>::type;
  T *y = static_cast<T *>(g.y);
  if constexpr (DT == kF32) y += static_cast<size_t>(blockIdx.y) * g.M * g.N;
  if (g.N % 8 == 0) {
    // 32 tokens at a time through LDS, so that neighbouring lanes store
    // neighbouring outputs: kChunk bytes of a row by kLanes lanes (8192 tokens 4096
    // -> 14336 279 us; straight from the registers, 32 bytes of a row by two
    // lanes, 287; in fp32, 14336 x 4096 over 8192 tokens, 273 and 294).
    constexpr int kSize = sizeof(T), kChunk = 64 * NB, kPitch = kChunk + 16, kLanes = kChunk / 16;
    constexpr int kBlocks = kChunk / (32 * kSize), kPer = 64 / kLanes;
    static_assert(sizeof(Buffer) >= GM * GN * 32 * kPitch, "a wave's rows");
    uint8_t *mine = reinterpret_cast<uint8_t *>(&q0) + wave * 32 * kPitch;
    const int at = lane % kLanes;
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j0 = 0; j0 < NB; j0 += kBlocks) {
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) place_block<DT>(mine + r * kPitch + 32 * kSize * j, h, acc[i][j0 + j]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const int n = col0 + wn + 32 * j0 + at * (16 / kSize);
#pragma unroll
        for (int p = 0; p < 32; p += kPer) {
          const int row = p + lane / kLanes, token = wm + 32 * i + row;
          const uint4 v = *reinterpret_cast<const uint4 *>(mine + row * kPitch + 16 * at);
          if (token < n_rows && n < g.N)
            *reinterpret_cast<uint4 *>(y + (static_cast<size_t>(i0) + token) * g.N + n) = v;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
  } else {
    // rows of y that start anywhere: value by value from the registers (2048 tokens
    // 4096 -> 4100 or 4097 in bf16 56 us; 4104, through LDS, 36; 4096 26)
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int token = wm + 32 * i + r;
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int n = col0 + wn + 32 * j + 8 * (k / 4) + 4 * h + k % 4;
          if (token < n_rows && n < g.N) y[(static_cast<size_t>(i0) + token) * g.N + n] = from_f32<DT>(acc[i][j][k]);
        }
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

template <int MB, int NB, int GM, int GN>
hipError_t launch_tiles(GemmArgs g, int dtype, int slices, hipStream_t s) {
  using Tl = Tile<MB, NB, GM, GN>;
  // grouped: every expert may end in a ragged tile
  const long tm = (static_cast<long>(g.M) + Tl::kM - 1) / Tl::kM + (g.E > 0 ? std::min(g.E, g.M) : 0);
  const long tn = (static_cast<long>(g.N) + Tl::kN - 1) / Tl::kN;
  if (tm * tn >= (1l << 24)) return hipErrorInvalidValue;   // a grid holds fewer than 2^32 threads
  g.tiles_m = static_cast<int>(tm);
  g.tiles_n = static_cast<int>(tn);
  const dim3 grid(static_cast<unsigned>(tm * tn), static_cast<unsigned>(slices)), block(Tl::kThreads);
#define LBQ_MX_GO(DT, GROUPED) \
  hipLaunchKernelGGL((mx_tile_kernel<MB, NB, GM, GN, DT, GROUPED>), grid, block, 0, s, g)
  if (g.E > 0) {   // in 16 bits
    if (dtype == kF16) LBQ_MX_GO(kF16, true);
    else if (dtype == kBF16) LBQ_MX_GO(kBF16, true);
    else return hipErrorInvalidValue;
  } else if (dtype == kF16) {
    LBQ_MX_GO(kF16, false);
  } else if (dtype == kBF16) {
    LBQ_MX_GO(kBF16, false);
  } else {
    LBQ_MX_GO(kF32, false);
  }
#undef LBQ_MX_GO
  return hipGetLastError();
}

// Which tile, and how many slices of K. Per 4096 of K, T tiles take about, in us:
// 256 x 256, one workgroup on a compute unit, 41 a round of 256; 128 x 128, two,
// 6 + 12 T / 256; 64 x 128, three, 6 + 6.6 T / 256 (T at least 256 in both). The
// least of them is taken. Measured at K = 4096 (64 x 128, 128 x 128, 256 x 256):
// 512 x 4096 12.7, 16.0, 34.1; 2048 x 4096 34, 28, 36; 400 x 28672 47, 44, 40;
// 4096 x 4096 59, 48, 43. Grouped, every expert's last tile is taken to be half
// full: 256 experts of 2048 x 2048, 64 rows each, 175, 191, 235; 8 of 4096 x 4096,
// 512 rows, 81, 73, 88; 8 of 28672 x 4096, 2048 rows, 2085, 1681, 1355. The starts
// in these costs do not grow with K, so other K shift the borders a little. Dense,
// K of 512, 1024, 2048, 8192 and 14336 at 512, 2048 and 4096 x 4096, 400 x 28672
// and 1000 x 8192: the tile taken is within 5 % of the best of the three. Grouped
// rows of long K would do better with larger tiles than the rule takes: 256 experts
// at 64 rows, K = 7168, 538 (64 x 128), 486, 565; 16 of 4096 at 128 rows, K =
// 14336, 196 (64 x 128), 192, 150; K = 2048 34.7, 36.3, 34.2. Dense with
// fewer tiles of the smallest kind than half the compute units: K in slices of
// at least 1024.
struct Plan {
  int bm, bn, slices;
};
Plan plan_tiles(const MxGemm &p) {
  auto tiles = [&](int bm, int bn) {
    const long tm = p.E > 0 ? std::max<long>(p.M / bm + p.E / 2, std::min(p.E, p.M))
                            : (static_cast<long>(p.M) + bm - 1) / bm;
    return tm * ((static_cast<long>(p.N) + bn - 1) / bn);
  };
  auto per_unit = [&](int bm, int bn) { return std::max(1.0, tiles(bm, bn) / 256.0); };
  const double big = 41 * static_cast<double>((tiles(256, 256) + 255) / 256);
  const double mid = 6 + 12 * per_unit(128, 128), small = 6 + 6.6 * per_unit(64, 128);
  if (big <= mid && big <= small) return {256, 256, 1};
  if (mid <= small) return {128, 128, 1};
  Plan r{64, 128, 1};
  if (p.E == 0)
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
  if (r.bm == 256) e = launch_tiles<4, 4, 2, 2>(g, dtype, r.slices, s);
  else if (r.bm == 128) e = launch_tiles<2, 2, 2, 2>(g, dtype, r.slices, s);
  else e = launch_tiles<1, 2, 2, 2>(g, dtype, r.slices, s);
  if (e != hipSuccess || r.slices == 1) return e;
  const long n = static_cast<long>(p.M) * p.N;
  hipLaunchKernelGGL(mx_sum_kernel, dim3(static_cast<unsigned>(std::min<long>((n + 255) / 256, 2048))), dim3(256), 0, s,
                     static_cast<const float *>(p.scratch), r.slices, n, p.dtype, p.y);
  return hipGetLastError();
}

}  // namespace lbq
