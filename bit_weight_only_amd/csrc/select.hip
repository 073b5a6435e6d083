// Expert selection: router logits to each token's experts and their weights,
// with softmax or sigmoid scores, a bias for choosing, groups of experts and
// renormalised weights; and the gradient of the weights.
//
//   p_e = exp(l_e) / sum exp(l)  or  1 / (1 + exp(-l_e)),   c_e = p_e + b_e
//
// picks go by c (by l where there is neither a bias nor groups: p rises with
// l), decided as 64-bit arithmetic decides it; weights come from p.
#include "device.h"
#include "kernels.h"
#include "mxfp4.h"

namespace lbq {

namespace {

using namespace mxfp4;

constexpr int kSelectThreads = 256, kWaves = kSelectThreads / 64;
constexpr double kNone = -__builtin_inf();

template <class T, class F>
__device__ __forceinline__ T wave_all(T v, F f) {
  for (int x = 32; x > 0; x /= 2) v = f(v, __shfl_xor(v, x));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
  return wave_all(v, [](double a, double b) { return a + b; });
}
__device__ __forceinline__ double wave_max(double v) {
  return wave_all(v, [](double a, double b) { return a > b ? a : b; });
}
__device__ __forceinline__ int wave_min(int v) {
  return wave_all(v, [](int a, int b) { return a < b ? a : b; });
}

// One wavefront per token, expert e = lane + 64 i.
template <int DT, int PER>
__global__ void __launch_bounds__(kSelectThreads) moe_select_kernel(MoeSelect r, const void *__restrict__ logits, int M,
                                                                    const float *__restrict__ bias,
                                                                    int32_t *__restrict__ ids,
                                                                    float *__restrict__ weights) {
  using T = typename Elem<DT>::type;
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (t >= M) return;
  const T *row = static_cast<const T *>(logits) + static_cast<size_t>(t) * r.E;
  double l[PER], p[PER], c[PER];
  double top = kNone;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    const float v = e < r.E ? to_f32<DT>(row[e]) : -INFINITY;
    l[i] = v > -INFINITY ? fmin(static_cast<double>(v), 3.4028234663852886e38) : kNone;   // NaN: none
    top = fmax(top, l[i]);
  }
  top = wave_max(top);
  double sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (r.score == kSoftmax) {
      p[i] = l[i] > kNone ? exp(l[i] - top) : 0.;
      sum += p[i];
    } else {
      p[i] = l[i] > kNone ? 1. / (1. + exp(-l[i])) : 0.;
    }
  }
  if (r.score == kSoftmax) {
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < PER; ++i) p[i] = sum > 0 ? p[i] / sum : 0.;
  }
  const bool by_logit = !bias && r.groups == 1;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    const float b = bias && e < r.E ? bias[e] : 0.f;
    c[i] = l[i] > kNone && b > -INFINITY ? (by_logit ? l[i] : p[i] + b) : kNone;
  }
  if (r.groups > 1) {
    const int each = r.E / r.groups;
    // lane g's group's value, 64 groups at a time, kept as a bit of `chosen`
    double value[PER];   // group lane + 64 i
#pragma unroll
    for (int i = 0; i < PER; ++i) value[i] = kNone;
    for (int g = 0; g < r.groups; ++g) {
      double first = kNone, v = kNone;
      int at = -1;
      for (int n = 0; n < r.group_picks; ++n) {
        double best = kNone;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int e = lane + 64 * i;
          if (e / each == g && e < r.E && e != at) best = fmax(best, c[i]);
        }
        best = wave_max(best);
        if (n == 0) {
          first = v = best;
          int mine = r.E;
#pragma unroll
          for (int i = PER - 1; i >= 0; --i) {
            const int e = lane + 64 * i;
            if (e < r.E && e / each == g && c[i] == first) mine = e;
          }
          at = wave_min(mine);
        } else if (best > kNone) {
          v = first + best;
        }
      }
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (lane + 64 * i == g) value[i] = v;
    }
    uint32_t chosen = 0;   // bit i: group lane + 64 i
    for (int n = 0; n < r.top_groups; ++n) {
      double best = kNone;
#pragma unroll
      for (int i = 0; i < PER; ++i) best = fmax(best, value[i]);
      best = wave_max(best);
      if (best == kNone) break;
      int mine = 64 * PER;
#pragma unroll
      for (int i = PER - 1; i >= 0; --i)
        if (value[i] == best) mine = lane + 64 * i;
      mine = wave_min(mine);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (lane + 64 * i == mine) {
          value[i] = kNone;
          chosen |= 1u << i;
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int g = min(lane + 64 * i, r.E - 1) / each;
      bool kept = false;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const uint32_t o = __shfl(chosen, g & 63);
        if (j == (g >> 6)) kept = (o >> j) & 1;
      }
      if (!kept) c[i] = kNone;
    }
  }
  // lane j keeps pick j's score
  double mine = 0, total = 0;
  int id = -1;
  for (int j = 0; j < r.top_k; ++j) {
    double best = kNone;
#pragma unroll
    for (int i = 0; i < PER; ++i) best = fmax(best, c[i]);
    best = wave_max(best);
    if (best == kNone) break;
    int e = 64 * PER;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i)
      if (c[i] == best) e = lane + 64 * i;
    e = wave_min(e);
    double s = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane + 64 * i == e) {
        s = p[i];
        c[i] = kNone;
      }
    s = __shfl(s, e & 63);
    total += s;
    if (lane == j) {
      mine = s;
      id = e;
    }
  }
  if (lane < r.top_k) {
    if (r.renormalise) mine = total > 0 ? mine / total : 0.;
    ids[static_cast<size_t>(t) * r.top_k + lane] = id;
    weights[static_cast<size_t>(t) * r.top_k + lane] = r.scale * static_cast<float>(mine);
  }
}

// d_logits of the weights' gradient: with S = sum of the picked p (renormalised) or
// 1, ds_j = scale (g_j - [renormalised] sum_i p_i g_i / S) / S, then the score's own
// derivative: sigmoid p (1 - p) ds, softmax p_e (ds_e - sum p ds).
template <int DT, int PER>
__global__ void __launch_bounds__(kSelectThreads) moe_select_backward_kernel(
    MoeSelect r, const float *__restrict__ d_w, const void *__restrict__ logits, int M,
    const int32_t *__restrict__ ids, void *__restrict__ d_logits) {
  using T = typename Elem<DT>::type;
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (t >= M) return;
  const T *row = static_cast<const T *>(logits) + static_cast<size_t>(t) * r.E;
  double l[PER], p[PER], ds[PER];
  double top = kNone;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    const float v = e < r.E ? to_f32<DT>(row[e]) : -INFINITY;
    l[i] = v > -INFINITY ? fmin(static_cast<double>(v), 3.4028234663852886e38) : kNone;
    top = fmax(top, l[i]);
    ds[i] = 0;
  }
  top = wave_max(top);
  double sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (r.score == kSoftmax) {
      p[i] = l[i] > kNone ? exp(l[i] - top) : 0.;
      sum += p[i];
    } else {
      p[i] = l[i] > kNone ? 1. / (1. + exp(-l[i])) : 0.;
    }
  }
  if (r.score == kSoftmax) {
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < PER; ++i) p[i] = sum > 0 ? p[i] / sum : 0.;
  }
  // the picks' scores and their sums
  double S = 0, dot = 0;
  for (int j = 0; j < r.top_k; ++j) {
    const int e = ids[static_cast<size_t>(t) * r.top_k + j];
    if (e < 0 || e >= r.E) continue;
    double s = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i == (e >> 6)) s = p[i];
    s = __shfl(s, e & 63);
    S += s;
    dot += s * d_w[static_cast<size_t>(t) * r.top_k + j];
  }
  const double inv = r.renormalise ? (S > 0 ? 1. / S : 0.) : 1.;
  for (int j = 0; j < r.top_k; ++j) {
    const int e = ids[static_cast<size_t>(t) * r.top_k + j];
    if (e < 0 || e >= r.E) continue;
    const double g = d_w[static_cast<size_t>(t) * r.top_k + j];
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane + 64 * i == e) ds[i] += r.scale * inv * (r.renormalise ? g - dot * inv : g);
  }
  double across = 0;
  if (r.score == kSoftmax) {
#pragma unroll
    for (int i = 0; i < PER; ++i) across += p[i] * ds[i];
    across = wave_sum(across);
  }
  T *out = static_cast<T *>(d_logits) + static_cast<size_t>(t) * r.E;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    double d = 0;
    if (l[i] > kNone) d = r.score == kSoftmax ? p[i] * (ds[i] - across) : ds[i] * p[i] * (1. / (1. + exp(l[i])));
    if (e < r.E) out[e] = from_f32<DT>(static_cast<float>(d));
  }
}

}  // namespace

#define LBQ_SELECT_PER(DT, KERNEL, ...)                                                         \
  do {                                                                                          \
    if (r.E <= 64) hipLaunchKernelGGL((KERNEL<DT, 1>), grid, block, 0, s, __VA_ARGS__);         \
    else if (r.E <= 256) hipLaunchKernelGGL((KERNEL<DT, 4>), grid, block, 0, s, __VA_ARGS__);   \
    else hipLaunchKernelGGL((KERNEL<DT, 16>), grid, block, 0, s, __VA_ARGS__);                  \
  } while (0)
#define LBQ_SELECT(KERNEL, ...)                                              \
  do {                                                                       \
    const dim3 grid((M + kWaves - 1) / kWaves), block(kSelectThreads);       \
    if (dtype == kF16) LBQ_SELECT_PER(kF16, KERNEL, __VA_ARGS__);            \
    else if (dtype == kBF16) LBQ_SELECT_PER(kBF16, KERNEL, __VA_ARGS__);     \
    else LBQ_SELECT_PER(kF32, KERNEL, __VA_ARGS__);                          \
  } while (0)

hipError_t launch_moe_select(const MoeSelect &r, const void *logits, int dtype, int M, const float *bias, int32_t *ids,
                             float *weights, hipStream_t s) {
  LBQ_SELECT(moe_select_kernel, r, logits, M, bias, ids, weights);
  return hipGetLastError();
}

hipError_t launch_moe_select_backward(const MoeSelect &r, const float *d_w, const void *logits, int dtype, int M,
                                      const int32_t *ids, void *d_logits, hipStream_t s) {
  LBQ_SELECT(moe_select_backward_kernel, r, d_w, logits, M, ids, d_logits);
  return hipGetLastError();
}

}  // namespace lbq
