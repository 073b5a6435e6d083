// Low-rank adapters of many requests beside a shared projection, and their
// gradients. Token t with adapter a = ids[t], scale s_a:
//
//   h_t = x_t A_a^T              y_t  = base_t + s_a h_t B_a^T
//   u_t = s_a dy_t B_a           dx_t = base_t + u_t A_a
//   dA_a = sum_t u_t^T x_t       dB_a = s_a sum_t dy_t^T h_t
//
// The sums over tokens run over the list of the adapter's tokens in the sorted
// order, so repeated calls give identical bits.
#include "device.h"
#include "kernels.h"
#include "mxfp4.h"

#include <algorithm>

namespace lbq {

namespace {

using namespace mxfp4;

constexpr int kThreads = 256;

__device__ __forceinline__ int adapter_of(const int32_t *ids, int t, int L) {
  const int a = ids[t];
  return a >= 0 && a < L ? a : -1;
}

// out[t][j] = scale sum_c x[t][c] w[a][j][c] (rows of w: r, columns C), one wave per (t, j)
template <int DT, bool T>
__global__ void __launch_bounds__(kThreads) adapters_down_kernel(const void *__restrict__ x, int C, int r,
                                                                 const void *__restrict__ w,
                                                                 const float *__restrict__ scales, int L,
                                                                 const int32_t *__restrict__ ids, float *out) {
  using E = typename Elem<DT>::type;
  const int t = blockIdx.x, lane = threadIdx.x & 63;
  const int a = adapter_of(ids, t, L);
  for (int j = threadIdx.x >> 6; j < r; j += kThreads / 64) {
    float s = 0;
    if (a >= 0) {
      const E *xr = static_cast<const E *>(x) + static_cast<size_t>(t) * C;
      const E *wr = static_cast<const E *>(w) + static_cast<size_t>(a) * r * C;
      for (int c = lane; c < C; c += 64)
        s = fmaf(to_f32<DT>(xr[c]), to_f32<DT>(wr[T ? static_cast<size_t>(c) * r + j : static_cast<size_t>(j) * C + c]), s);
    }
    for (int d = 32; d > 0; d /= 2) s += __shfl_xor(s, d);
    if (lane == 0) out[static_cast<size_t>(t) * r + j] = a >= 0 ? s * (scales ? scales[a] : 1.f) : 0.f;
  }
}

// y[t][c] = base[t][c] + scale sum_j h[t][j] w[a][j][c]
template <int DT, bool T>
__global__ void __launch_bounds__(kThreads) adapters_up_kernel(const float *__restrict__ h, int C, int r,
                                                               const void *__restrict__ w,
                                                               const float *__restrict__ scales, int L,
                                                               const int32_t *__restrict__ ids, const void *base,
                                                               void *y) {
  using E = typename Elem<DT>::type;
  const int t = blockIdx.x;
  const int a = adapter_of(ids, t, L);
  for (int c = blockIdx.y * kThreads + threadIdx.x; c < C; c += gridDim.y * kThreads) {
    float s = 0;
    if (a >= 0) {
      const E *wr = static_cast<const E *>(w) + static_cast<size_t>(a) * r * C;
      for (int j = 0; j < r; ++j)
        s = fmaf(h[static_cast<size_t>(t) * r + j],
                 to_f32<DT>(wr[T ? static_cast<size_t>(c) * r + j : static_cast<size_t>(j) * C + c]), s);
    }
    const size_t at = static_cast<size_t>(t) * C + c;
    const float b = base ? to_f32<DT>(static_cast<const E *>(base)[at]) : 0.f;
    static_cast<E *>(y)[at] = from_f32<DT>(a >= 0 ? fmaf(s, scales ? scales[a] : 1.f, b) : b);
  }
}

// out[a][j][c] (T: [a][c][j]) = scale sum over a's tokens of g[t][j] x[t][c]
template <int DT, bool T>
__global__ void __launch_bounds__(kThreads) adapters_grad_kernel(const float *__restrict__ g,
                                                                 const void *__restrict__ x, int M, int C, int r,
                                                                 const float *__restrict__ scales,
                                                                 const int32_t *__restrict__ offsets,
                                                                 const int32_t *__restrict__ perm, float *out) {
  using E = typename Elem<DT>::type;
  const int a = blockIdx.z, j = blockIdx.y;
  const int lo = min(max(offsets[a], 0), M), hi = min(max(offsets[a + 1], lo), M);
  for (int c = blockIdx.x * kThreads + threadIdx.x; c < C; c += gridDim.x * kThreads) {
    float s = 0;
    for (int i = lo; i < hi; ++i) {
      const int t = perm[i];
      if (t < 0 || t >= M) continue;
      s = fmaf(g[static_cast<size_t>(t) * r + j], to_f32<DT>(static_cast<const E *>(x)[static_cast<size_t>(t) * C + c]), s);
    }
    const size_t at = static_cast<size_t>(a) * r * C;
    out[at + (T ? static_cast<size_t>(c) * r + j : static_cast<size_t>(j) * C + c)] = scales ? s * scales[a] : s;
  }
}

}  // namespace

size_t adapters_ws_bytes(const AdapterArgs &g, bool backward) {
  return static_cast<size_t>(g.M) * g.r * 4;
}

bool adapters_forward_by_list(const AdapterArgs &) { return false; }

hipError_t launch_adapters_forward(const AdapterArgs &g, hipStream_t s) {
  float *h = g.h ? g.h : static_cast<float *>(g.scratch);
  const dim3 grid(g.M), up(g.M, std::min((g.N + kThreads - 1) / kThreads, 64)), block(kThreads);
#define GO(DT)                                                                                                       \
  hipLaunchKernelGGL((adapters_down_kernel<DT, false>), grid, block, 0, s, g.x, g.K, g.r, g.a, nullptr, g.L, g.ids, h); \
  hipLaunchKernelGGL((adapters_up_kernel<DT, true>), up, block, 0, s, h, g.N, g.r, g.b, g.scales, g.L, g.ids, g.base, g.y)
  if (g.dtype == kF16) { GO(kF16); } else { GO(kBF16); }
#undef GO
  return hipGetLastError();
}

hipError_t launch_adapters_backward(const AdapterArgs &g, hipStream_t s) {
  float *u = static_cast<float *>(g.scratch);
  const dim3 grid(std::max(g.M, 1)), block(kThreads);
  const int kb = std::min((g.K + kThreads - 1) / kThreads, 64), nb = std::min((g.N + kThreads - 1) / kThreads, 64);
#define GO(DT)                                                                                                      \
  if (g.M > 0) {                                                                                                    \
    hipLaunchKernelGGL((adapters_down_kernel<DT, true>), grid, block, 0, s, g.dy, g.N, g.r, g.b, g.scales, g.L, g.ids, u); \
    hipLaunchKernelGGL((adapters_up_kernel<DT, false>), dim3(g.M, kb), block, 0, s, u, g.K, g.r, g.a, nullptr, g.L, g.ids, g.base, g.y); \
  }                                                                                                                 \
  hipLaunchKernelGGL((adapters_grad_kernel<DT, false>), dim3(kb, g.r, g.L), block, 0, s, u, g.x, g.M, g.K, g.r, nullptr, g.offsets, g.perm, g.d_a); \
  hipLaunchKernelGGL((adapters_grad_kernel<DT, true>), dim3(nb, g.r, g.L), block, 0, s, g.h, g.dy, g.M, g.N, g.r, g.scales, g.offsets, g.perm, g.d_b)
  if (g.dtype == kF16) { GO(kF16); } else { GO(kBF16); }
#undef GO
  return hipGetLastError();
}

}  // namespace lbq
