// Products of MXFP4 tensors: y[i][n] = sum_k a[i][k] b[n][k], dense and grouped
// over experts, on v_mfma_scale_f32_32x32x64_f8f6f4 (both operands fp4, the
// E8M0 scales applied inside the instruction, fp32 accumulation).
//
// Operand layout of the instruction: lane (r, h), r = lane & 31, h = lane >> 5,
// holds the 32 values of row r, block h of the 64-long step (16 bytes) and that
// block's scale byte; result register i of lane (c, h) is row
// 8 (i / 4) + 4 h + i % 4, column c.
#include "device.h"
#include "kernels.h"
#include "mxfp4.h"

#include <algorithm>

namespace lbq {

namespace {

using namespace mxfp4;

typedef int v8i_t __attribute__((ext_vector_type(8)));
typedef float v16f_t __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;
constexpr int kTile = 128;   // rows and columns of a workgroup: four waves of 64 x 64

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
};

// 128 x 128 per workgroup, operands straight from memory (each lane's 16 bytes).
template <int DT, bool GROUPED>
__global__ void __launch_bounds__(kThreads) mx_gemm_kernel(GemmArgs g) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 31, h = lane >> 5;
  int i0 = blockIdx.y * kTile, n_rows = g.M - i0, e = 0;
  if constexpr (GROUPED) {
    const GroupTile t = find_tile(g.offsets, g.E, g.M, kTile, blockIdx.y);
    if (t.n == 0) return;
    i0 = t.i0;
    n_rows = t.n;
    e = t.e;
  }
  const int wm = (wave >> 1) * 64, wn = blockIdx.x * kTile + (wave & 1) * 64;
  const uint8_t *pa[2], *pb[2];
  const uint32_t *sa[2], *sb[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    // rows past the end repeat the last one; their results are not stored
    int ia = i0 + min(wm + 32 * t + r, n_rows - 1);
    if constexpr (GROUPED)
      if (g.perm) ia = g.perm[ia] / g.top_k;
    ia = min(max(ia, 0), g.a_rows - 1);
    const int ib = e * g.N + min(wn + 32 * t + r, g.N - 1);
    pa[t] = g.a_codes + static_cast<size_t>(ia) * (g.K / 2) + 16 * h;
    pb[t] = g.b_codes + static_cast<size_t>(ib) * (g.K / 2) + 16 * h;
    sa[t] = g.a_scales + ia;
    sb[t] = g.b_scales + ib;
  }
  v16f_t acc[2][2];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[0][0][i] = acc[0][1][i] = acc[1][0][i] = acc[1][1][i] = 0.f;
  for (int kg = 0; kg < g.K / kGroup; ++kg) {
    int va[2], vb[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      va[t] = static_cast<int>(sa[t][static_cast<size_t>(kg) * g.a_rows] >> (8 * h));
      vb[t] = static_cast<int>(sb[t][static_cast<size_t>(kg) * g.b_rows] >> (8 * h));
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      v8i_t fa[2], fb[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        fa[t] = operand(*reinterpret_cast<const uint4 *>(pa[t] + 64 * static_cast<size_t>(kg) + 32 * s));
        fb[t] = operand(*reinterpret_cast<const uint4 *>(pb[t] + 64 * static_cast<size_t>(kg) + 32 * s));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = s == 0 ? __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[i], fb[j], acc[i][j], 4, 4, 0, va[i],
                                                                              0, vb[j])
                             : __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[i], fb[j], acc[i][j], 4, 4, 2, va[i],
                                                                              2, vb[j]);
    }
  }
  using T = typename Elem<DT>::type;
  T *y = static_cast<T *>(g.y);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int row = wm + 32 * i + 8 * (k / 4) + 4 * h + k % 4, n = wn + 32 * j + r;
        if (row < n_rows && n < g.N) y[static_cast<size_t>(i0 + row) * g.N + n] = from_f32<DT>(acc[i][j][k]);
      }
}

}  // namespace

hipError_t launch_mx_gemm(const MxGemm &p, hipStream_t s) {
  GemmArgs g{};
  g.a_codes = static_cast<const uint8_t *>(p.a_codes);
  g.a_scales = static_cast<const uint32_t *>(p.a_scales);
  g.b_codes = static_cast<const uint8_t *>(p.b_codes);
  g.b_scales = static_cast<const uint32_t *>(p.b_scales);
  g.y = p.y;
  g.a_rows = p.a_rows;
  g.b_rows = p.E > 0 ? p.E * p.N : p.N;
  g.M = p.M;
  g.N = p.N;
  g.K = p.K;
  g.offsets = p.offsets;
  g.perm = p.perm;
  g.E = p.E;
  g.top_k = p.top_k;
  // grouped: every expert may end in a ragged tile
  const long tiles = (static_cast<long>(p.M) + kTile - 1) / kTile + (p.E > 0 ? std::min(p.E, p.M) : 0);
  const dim3 grid((p.N + kTile - 1) / kTile, static_cast<unsigned>(tiles));
#define LBQ_MX_GO(DT)                                                                             \
  if (p.E > 0) hipLaunchKernelGGL((mx_gemm_kernel<DT, true>), grid, dim3(kThreads), 0, s, g);     \
  else hipLaunchKernelGGL((mx_gemm_kernel<DT, false>), grid, dim3(kThreads), 0, s, g)
  if (p.dtype == kF16) {
    LBQ_MX_GO(kF16);
  } else if (p.dtype == kBF16) {
    LBQ_MX_GO(kBF16);
  } else {
    LBQ_MX_GO(kF32);
  }
#undef LBQ_MX_GO
  return hipGetLastError();
}

size_t mx_gemm_scratch_bytes(const MxGemm &) { return 0; }

}  // namespace lbq
