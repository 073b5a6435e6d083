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

#include <algorithm>

namespace lbq {

namespace {

using namespace mxfp4;

constexpr int kSelectThreads = 256, kWaves = kSelectThreads / 64;
constexpr double kNone = -__builtin_inf();
// Softmax scores of logits this much below their row's largest are 0 in 64 bits.
constexpr double kNothing = -745.;
// Sigmoids from this logit down are 0 in 64 bits: exp(-l) is infinite there.
constexpr float kNoSigmoid = -709.7827f;

// Value of the lane N further round in its row of 16.
template <int N>
__device__ __forceinline__ uint32_t turned(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x120 + N, 0xF, 0xF, false));
}
template <int N>
__device__ __forceinline__ float turned(float v) {
  return __uint_as_float(turned<N>(__float_as_uint(v)));
}
template <int N>
__device__ __forceinline__ double turned(double v) {
  return __hiloint2double(static_cast<int>(turned<N>(static_cast<uint32_t>(__double2hiint(v)))),
                          static_cast<int>(turned<N>(static_cast<uint32_t>(__double2loint(v)))));
}
template <int X>
__device__ __forceinline__ float crossed(float v) {
  return __uint_as_float(xor_lane_u32<X>(__float_as_uint(v)));
}
template <int X>
__device__ __forceinline__ double crossed(double v) {
  return __hiloint2double(static_cast<int>(xor_lane_u32<X>(static_cast<uint32_t>(__double2hiint(v)))),
                          static_cast<int>(xor_lane_u32<X>(static_cast<uint32_t>(__double2loint(v)))));
}
// Over the LANES lanes of a token, in each of them.
template <int LANES, class T, class F>
__device__ __forceinline__ T row_all(T v, F f) {
  v = f(v, turned<8>(v));
  v = f(v, turned<4>(v));
  v = f(v, turned<2>(v));
  v = f(v, turned<1>(v));
  if constexpr (LANES == 64) {
    v = f(v, crossed<16>(v));
    v = f(v, crossed<32>(v));
  }
  return v;
}
// Token t in 64 bits, by a whole wavefront: for the rare token whose order 32 bits leave
// open (and for more groups than the fast form takes). cs, gs: LDS for E choice
// values and the groups' values.
template <int DT>
__device__ __forceinline__ void select_exactly(const MoeSelect &r, const void *__restrict__ logits, int t,
                                               const float *__restrict__ bias, double *cs, double *gs,
                                               int32_t *__restrict__ ids, float *__restrict__ weights) {
  using T = typename Elem<DT>::type;
  const int lane = threadIdx.x & 63;
  const T *row = static_cast<const T *>(logits) + static_cast<size_t>(t) * r.E;
  auto logit = [&](int e) {   // NaN: none
    const float v = to_f32<DT>(row[e]);
    return v > -INFINITY ? static_cast<double>(fminf(v, 3.4028234663852886e38f)) : kNone;
  };
  double top = kNone, sum = 0.;
  if (r.score == kSoftmax) {
    for (int e = lane; e < r.E; e += 64) top = fmax(top, logit(e));
    top = row_all<64>(top, [](double a, double b) { return fmax(a, b); });
    for (int e = lane; e < r.E; e += 64) sum += logit(e) > kNone ? exp(logit(e) - top) : 0.;
    sum = row_all<64>(sum, [](double a, double b) { return a + b; });
  }
  auto score = [&](double l) {
    if (!(l > kNone)) return 0.;
    return r.score == kSigmoid ? 1. / (1. + exp(-l)) : exp(l - top) / sum;
  };
  const bool by_logit = !bias && r.groups == 1;
  for (int e = lane; e < r.E; e += 64) {
    const double l = logit(e);
    const float b = bias ? bias[e] : 0.f;
    cs[e] = l > kNone && b > -INFINITY ? (by_logit ? l : score(l) + b) : kNone;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (r.groups > 1) {
    const int each = r.E / r.groups;
    for (int g = lane; g < r.groups; g += 64) {
      double first = kNone, second = kNone;
      for (int i = 0; i < each; ++i) {
        const double x = cs[g * each + i];
        second = fmax(second, fmin(first, x));
        first = fmax(first, x);
      }
      gs[g] = r.group_picks == 2 && second > kNone ? first + second : first;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    for (int g = lane; g < r.groups; g += 64) {
      const double x = gs[g];
      int rank = 0;
      for (int o = 0; o < r.groups; ++o) rank += gs[o] > x || (gs[o] == x && o < g);
      if (rank >= r.top_groups)
        for (int i = 0; i < each; ++i) cs[g * each + i] = kNone;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  // lane j keeps pick j
  int id = -1;
  for (int j = 0; j < r.top_k; ++j) {
    double best = kNone;
    int at = r.E;
    for (int e = lane; e < r.E; e += 64)
      if (cs[e] > best) {
        best = cs[e];
        at = e;
      }
    const double all = row_all<64>(best, [](double a, double b) { return fmax(a, b); });
    // the lowest of those that have it: as a float, exact below 2^24
    at = static_cast<int>(row_all<64>(best == all ? static_cast<float>(at) : 1e6f, [](float a, float b) { return fminf(a, b); }));
    if (at >= r.E) break;
    if (lane == j) id = at;
    if (lane == 0) cs[at] = kNone;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  double mine = id >= 0 ? score(logit(id)) : 0.;
  if (r.renormalise && r.score == kSoftmax) {
    // the ratio of scores that keep few bits themselves
    const double l = id >= 0 ? logit(id) : kNone;
    const double most = row_all<64>(l, [](double a, double b) { return fmax(a, b); });
    mine = l - top > kNothing ? exp(l - most) : 0.;
  }
  const double total = row_all<64>(mine, [](double a, double b) { return a + b; });
  if (lane < r.top_k) {
    if (r.renormalise) mine = total > 0. ? mine / total : 0.;
    ids[static_cast<size_t>(t) * r.top_k + lane] = id;
    weights[static_cast<size_t>(t) * r.top_k + lane] = r.scale * static_cast<float>(mine);
  }
}

// ------------------------------------------------------------------ rows of lanes

// LANES lanes a token, V logits a lane in pieces of 16 bytes (V = 4: of four): a
// lane's value i is expert first(i / P) + i % P. A piece that would reach past the
// last expert starts earlier; what it has twice is left out.
template <int DT, int LANES, int V>
struct Row {
  using T = typename Elem<DT>::type;
  static constexpr int P = V == 4 ? 4 : 16 / sizeof(T), kPieces = V / P;
  float v[V];
  static __device__ __forceinline__ int expert(int i, int lane) { return (i / P * LANES + lane) * P + i % P; }
  __device__ __forceinline__ void load(const T *row, int E, int lane) {
    struct __attribute__((packed, aligned(sizeof(T)))) Piece {
      T v[P];
    };
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int e = (k * LANES + lane) * P, from = min(e, E - P);
      Piece p;
      if (E >= P) {
        p = *reinterpret_cast<const Piece *>(row + from);
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) p.v[i] = row[min(e + i, E - 1)];
      }
      const int skip = E >= P ? e - from : 0;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        // value i is expert e + i: at i + skip of the piece
        T x = p.v[i];
        if (skip > 0) {
#pragma unroll
          for (int j = 0; j < P; ++j)
            if (j == i + skip) x = p.v[j];
        }
        // NaN is none
        v[k * P + i] = fminf(fmaxf(to_f32<DT>(x), -INFINITY), 3.4028234663852886e38f);
      }
      if (E < LANES * V) {   // experts past the last: none
#pragma unroll
        for (int i = 0; i < P; ++i) v[k * P + i] = e + i < E ? v[k * P + i] : -INFINITY;
      }
    }
  }
};

template <int LANES>
__device__ __forceinline__ float row_max(float v) {
  return row_all<LANES>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
  return row_all<LANES>(v, [](float a, float b) { return a + b; });
}

// A choice value and its expert as one double that orders like the pair, larger
// values first and of equal ones the lower expert: the whole number (value's order
// << 10 | 1023 - expert) added to 2^52. One instruction compares it. What is below
// kFirst is the value -infinity: none.
__device__ __forceinline__ double pair_of(float c, int e) {
  const uint32_t b = __float_as_uint(c + 0.f);   // -0 as 0
  const uint32_t o = b ^ (static_cast<uint32_t>(static_cast<int>(b) >> 31) | 0x80000000u);
  return __hiloint2double(static_cast<int>(0x43300000u | o >> 22), static_cast<int>(o << 10 | (1023u - e)));
}
constexpr double kFirst = 4503599627370496. + 8388608. * 1024.;   // 2^52 + (0x00800000 << 10)
__device__ __forceinline__ int expert_of(double d) { return 1023 - (__double2loint(d) & 1023); }
__device__ __forceinline__ float value_of(double d) {
  const uint32_t o = static_cast<uint32_t>(__double2hiint(d)) << 22 | static_cast<uint32_t>(__double2loint(d)) >> 10;
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
template <int LANES>
__device__ __forceinline__ double row_best(double v) {
  return row_all<LANES>(v, [](double a, double b) { return __builtin_fmax(a, b); });
}

// Larger first: an odd-even merge network.
template <int V>
__device__ __forceinline__ void sort_down(double (&v)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const double a = v[i + j], b = v[i + j + k];
            v[i + j] = __builtin_fmax(a, b);
            v[i + j + k] = __builtin_fmin(a, b);
          }
}

// A score times exp(-top): softmax up to its sum, sigmoid for top <= 0. Scores of one top
// keep their ratio where fp32 does not hold them themselves.
__device__ __forceinline__ float score_of(float l, int score, float top) {
  if (score == kSoftmax) return expf(l - top);
  const float one = __builtin_amdgcn_rcpf(1.f + expf(-fabsf(l)));
  return l > 0.f ? one : expf(l - top) * one;
}

// The same for the order alone: the argument's rounding counts for little, since p falls
// faster than it grows (x p (1 - p) and x exp(-x) stay below 0.4).
__device__ __forceinline__ float rough_score(float l, int score, float top) {
  constexpr float kLog2E = 1.44269504f;
  if (score == kSigmoid) return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2E * l));
  return __builtin_amdgcn_exp2f(kLog2E * (l - top));
}

constexpr int kMostGroups = 64;

// Each lane sorts its values once; then the heads of the lanes' lists are compared,
// and the winner's next value comes from LDS.
//
// 32 bits decide, but where two neighbours among the picks, or the last pick and
// the next, or the last group kept and the next, lie nearer than 32 bits can tell:
// then the token is done again in 64. In units u = 2^-24: a sigmoid is off by at most
// 4 u (exp's argument 0.5, exp 0.5, the sum 1, the reciprocal 2) and the sum with the
// bias by u (1 + |b|), so that a difference is off by 10 u + 2 u |b|; a softmax by 4 u of the
// row's largest score, and all of them together by their sum's up to 24 u; `near` is
// twice the one and more than the other.
//
// What bounds it is instructions: (top_k + 1) rounds, for 4 tokens at once with 16 lanes
// a token (131072 tokens of 256 experts, 8 picks, sigmoid with bias: 105 us, 286
// instructions a token, 0.7 TB/s). Few tokens take a wavefront each, whose lists are
// shorter: 2048 tokens of 256 experts, bf16, softmax 5.9 us against 6.8, sigmoid with bias
// 11.6 and 13.5, that in groups 16.9 and 19.0; 4096 tokens 7.8 and 6.8, 14.0 and 13.9, 19.5
// and 19.2 (32 tokens 5.4 us).
template <int DT, int LANES, int V>
__global__ void __launch_bounds__(kSelectThreads, 3) moe_select_kernel(MoeSelect r, const void *__restrict__ logits, int M,
                                                                    const float *__restrict__ bias,
                                                                    int32_t *__restrict__ ids,
                                                                    float *__restrict__ weights) {
  using T = typename Elem<DT>::type;
  using R = Row<DT, LANES, V>;
  constexpr int kTokens = 64 / LANES;   // of a wavefront
  __shared__ double lists[kWaves][V * 64];
  constexpr int kPicks = kMoeMaxTopK + 2;
  __shared__ double picks[kWaves][kTokens * kPicks > kMostGroups ? kTokens * kPicks : kMostGroups];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & (LANES - 1), mine = (threadIdx.x & 63) / LANES;
  double *list = lists[wave] + (threadIdx.x & 63);
  double *pick = picks[wave] + mine * kPicks;
  const bool by_logit = !bias && r.groups == 1;
  const bool whole = r.score == kSoftmax && (!by_logit || !r.renormalise);   // all scores of a row are needed
  float b[V], most = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = R::expert(i, lane);
    b[i] = bias && e < r.E ? bias[e] : 0.f;
    b[i] = b[i] > -INFINITY ? b[i] : -INFINITY;
    if (fabsf(b[i]) < INFINITY) most = fmaxf(most, fabsf(b[i]));
  }
  most = row_max<LANES>(most);
  const int each = r.E / r.groups;
  const uint32_t inverse = ((1u << 20) + each - 1) / each;   // e / each = e inverse >> 20 for e < 1024
  for (int t0 = (blockIdx.x * kWaves + wave) * kTokens; t0 < M; t0 += gridDim.x * kWaves * kTokens) {
    const int t = min(t0 + mine, M - 1);
    const T *row = static_cast<const T *>(logits) + static_cast<size_t>(t) * r.E;
    // (a number that the compiler does not know to be the same every time: it would
    // keep what follows from it, a register or a mask per value)
    int here = lane;
    asm volatile("" : "+v"(here));
    R l;
    l.load(row, r.E, here);
    float top = 0.f, inv = 1.f;
    if (r.score == kSoftmax) {
      top = -INFINITY;
#pragma unroll
      for (int i = 0; i < V; ++i) top = fmaxf(top, l.v[i]);
      top = row_max<LANES>(top);
    }
    float c[V];
    if (by_logit) {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = l.v[i];
    }
    if (whole || !by_logit) {
      // what is none has a score of 0 by itself (or, with nothing else there, NaN)
      float p[V];
      if (r.score == kSigmoid) {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = rough_score(l.v[i], kSigmoid, 0.f);
      } else {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          p[i] = rough_score(l.v[i], kSoftmax, top);
          sum += p[i];
        }
        sum = row_sum<LANES>(sum);
        inv = sum > 0.f ? 1.f / sum : 0.f;
      }
      if (!by_logit) {
        // (a bias of -infinity stays)
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = l.v[i] > -INFINITY ? fmaf(p[i], inv, b[i]) : -INFINITY;
      }
    }
    const float near = (r.score == kSoftmax ? 0x1p-18f * inv : 0x1.4p-20f) + 0x1p-22f * most;
    bool open = false;
    if (r.groups > 1) {
      // the choice values in LDS; a lane per group adds up its largest
      float *cs = reinterpret_cast<float *>(lists[wave]) + mine * (LANES * V);
#pragma unroll
      for (int i = 0; i < V; ++i) cs[R::expert(i, here)] = c[i];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      float *gs = reinterpret_cast<float *>(lists[wave]) + 64 * V + mine * kMostGroups;
      for (int g = lane; g < r.groups; g += LANES) {
        float first = -INFINITY, second = -INFINITY;
        for (int i = 0; i < each; ++i) {
          const float x = cs[g * each + i];
          second = fmaxf(second, fminf(first, x));
          first = fmaxf(first, x);
        }
        gs[g] = r.group_picks == 2 && second > -INFINITY ? first + second : first;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      // a group's rank; the last one kept and the next
      float last = -INFINITY, next = -INFINITY;
      uint64_t kept = 0;
      for (int g = lane; g < r.groups; g += LANES) {
        const float x = gs[g];
        int rank = 0;
        for (int o = 0; o < r.groups; ++o) {
          const float y = gs[o];
          rank += y > x || (y == x && o < g);
        }
        if (rank < r.top_groups && x > -INFINITY) kept |= 1ull << g;
        if (rank == r.top_groups - 1) last = x;
        if (rank == r.top_groups) next = x;
      }
      last = row_max<LANES>(last);
      next = row_max<LANES>(next);
      open = next > -INFINITY && !(last - next > 2.f * near);
      uint32_t lo = static_cast<uint32_t>(kept), hi = static_cast<uint32_t>(kept >> 32);
#pragma unroll
      for (int d = 1; d < LANES; d *= 2) {
        lo |= __shfl_xor(lo, d);
        hi |= __shfl_xor(hi, d);
      }
      kept = static_cast<uint64_t>(hi) << 32 | lo;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t g = static_cast<uint32_t>(R::expert(i, here)) * inverse >> 20;
        if (!(kept >> (g & 63) & 1)) c[i] = -INFINITY;
      }
    }
    double s[V];
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = pair_of(c[i], R::expert(i, here));
    sort_down<V>(s);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 2; i < V; ++i) list[64 * i] = s[i];
    // a lane's next value is there when the one before it wins
    double head = s[0], next = V > 1 ? s[V > 1 ? 1 : 0] : 0.;
    const double *after = list + 128;
    int left = V - 2;
    // one round more than picks, for the one that was not taken
    for (int j = 0; j < r.top_k + !by_logit; ++j) {
      const double best = row_best<LANES>(head);
      if (lane == 0) pick[j] = best;
      if (head == best) {
        head = next;
        next = left > 0 ? *after : 0.;
        after += 64;
        --left;
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    float p[2] = {0.f, 0.f}, x[2] = {-INFINITY, -INFINITY}, total = 0.f;
    int id[2] = {-1, -1};
#pragma unroll
    for (int n = 0; n < (LANES == 16 ? 2 : 1); ++n) {
      const int j = lane + LANES * n;
      if (j >= r.top_k || pick[j] < kFirst) continue;
      id[n] = expert_of(pick[j]);
      x[n] = fminf(to_f32<DT>(row[id[n]]), 3.4028234663852886e38f);
      if (!by_logit && pick[j + 1] >= kFirst && !(value_of(pick[j]) - value_of(pick[j + 1]) > near)) {
        // as near as that, but for the same logit and bias
        const int o = expert_of(pick[j + 1]);
        const float y = fminf(to_f32<DT>(row[o]), 3.4028234663852886e38f);
        open = open || x[n] != y || (bias && bias[id[n]] != bias[o]);
      }
    }
    // a ratio is taken relative to the largest pick, whose score can be a small one: a sigmoid
    // far below zero, a softmax that a bias keeps far below the row's largest (64 bits
    // know where such scores end)
    float from = top;
    if (r.renormalise && !(r.score == kSoftmax && by_logit)) {
      const float most = row_max<LANES>(fmaxf(x[0], x[1]));
      from = r.score == kSoftmax ? most : fminf(most, 0.f);
      open = open || (most > -INFINITY && top - from > 600.f);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      if (id[n] >= 0) p[n] = score_of(x[n], r.score, from);
      total += p[n];
    }
    total = row_sum<LANES>(total);
    const float factor = r.scale * (!r.renormalise ? inv : total > 0.f ? 1.f / total : 0.f);
    const uint64_t opens = __ballot(open);
    constexpr uint64_t kRow = LANES == 64 ? ~0ull : (1ull << (LANES & 63)) - 1;
    if (t0 + mine < M && !(opens >> (mine * LANES) & kRow)) {
#pragma unroll
      for (int n = 0; n < (LANES == 16 ? 2 : 1); ++n) {
        const int j = lane + LANES * n;
        if (j >= r.top_k) continue;
        ids[static_cast<size_t>(t) * r.top_k + j] = id[n];
        weights[static_cast<size_t>(t) * r.top_k + j] = p[n] * factor;
      }
    }
    for (int n = 0; n < kTokens; ++n)
      if (t0 + n < M && (opens >> (n * LANES) & kRow))
        select_exactly<DT>(r, logits, t0 + n, bias, lists[wave], picks[wave], ids, weights);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

// All tokens in 64 bits: for more than kMostGroups groups, a bit each of a mask in the
// fast form.
template <int DT>
__global__ void __launch_bounds__(kSelectThreads) moe_select_exact_kernel(MoeSelect r, const void *__restrict__ logits,
                                                                          int M, const float *__restrict__ bias,
                                                                          int32_t *__restrict__ ids,
                                                                          float *__restrict__ weights) {
  __shared__ double cs[kWaves][kMoeMaxExperts], gs[kWaves][kMoeMaxExperts];
  const int wave = threadIdx.x >> 6, t = blockIdx.x * kWaves + wave;
  if (t < M) select_exactly<DT>(r, logits, t, bias, cs[wave], gs[wave], ids, weights);
}

// ------------------------------------------------------------------ gradient

// The largest of E <= 16 V logits, NaN being none, in each of a token's 16 lanes. All
// loads are under way at once; a piece that would reach past the last starts earlier.
template <int DT, int V>
__device__ __forceinline__ float row_top(const typename Elem<DT>::type *row, int E, int lane) {
  using T = typename Elem<DT>::type;
  constexpr int P = 16 / sizeof(T), kPieces = (V + P - 1) / P;
  struct __attribute__((packed, aligned(sizeof(T)))) Piece {
    T v[P];
  };
  float top = -INFINITY;
  if (E >= P) {
    Piece p[kPieces];
#pragma unroll
    for (int k = 0; k < kPieces; ++k)
      if (k * 16 * P < E) p[k] = *reinterpret_cast<const Piece *>(row + min((k * 16 + lane) * P, E - P));
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      if (k * 16 * P >= E) continue;
#pragma unroll
      for (int i = 0; i < P; ++i) top = fmaxf(top, to_f32<DT>(p[k].v[i]));
    }
  } else {
    top = fmaxf(top, to_f32<DT>(row[min(lane, E - 1)]));
  }
  return fminf(row_max<16>(top), 3.4028234663852886e38f);
}

// d_logits of the weights' gradient: with S = sum of the picked p (renormalised) or
// 1, ds_j = scale (g_j - [renormalised] sum_i p_i g_i / S) / S, then the score's own
// derivative: sigmoid p (1 - p) ds, softmax p_e (ds_e - sum p ds). With renormalised
// softmax the last sum is zero, and the logits that were not picked fall out of it: so
// but for plain softmax a token's row is zeros and a few values. What bounds it then is
// writing the rows.
//
// Sigmoid, of whose logits only the picked are read: 131072 rows of 256 bf16 values 24.8
// us (67 MB written, parts of as much read).
// 16 lanes a token; the row is put together in LDS, slot after slot, so that an expert
// named twice gets both.
//
// Renormalised softmax takes the picks relative to their largest, and reads the whole row
// for the largest there: what 64 bits hold as 0 has no weight, and no gradient (131072
// rows of 256 bf16 values 29.9 us; 24.1 without that): RATIO, a kernel of its own, since the
// others are a microsecond slower with the code for it.
template <int DT, int V, bool RATIO>
__global__ void __launch_bounds__(kSelectThreads) moe_select_backward_kernel(
    MoeSelect r, const float *__restrict__ d_w, const void *logits, int M, const int32_t *__restrict__ ids,
    void *d_logits) {
  using T = typename Elem<DT>::type;
  constexpr int kLanes = 16, kTokens = 4, kRow = kLanes * V;   // E <= kRow
  __shared__ float rows[kWaves][kTokens][kRow];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 15, mine = (threadIdx.x & 63) / kLanes;
  const bool dense = r.score == kSoftmax && !r.renormalise;
  float *d = rows[wave][mine];
  for (int t0 = (blockIdx.x * kWaves + wave) * kTokens; t0 < M; t0 += gridDim.x * kWaves * kTokens) {
    const int t = min(t0 + mine, M - 1);
    const T *row = static_cast<const T *>(logits) + static_cast<size_t>(t) * r.E;
    auto logit = [&](int e) {   // NaN: none
      const float v = to_f32<DT>(row[e]);
      return v > -INFINITY ? fminf(v, 3.4028234663852886e38f) : -INFINITY;
    };
    float most = -INFINITY;
    if constexpr (RATIO) most = row_top<DT, V>(row, r.E, lane);
    int id[2];
    float l[2], g[2], top = -INFINITY;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int j = lane + kLanes * n;
      id[n] = j < r.top_k ? ids[static_cast<size_t>(t) * r.top_k + j] : -1;
      if (id[n] < 0 || id[n] >= r.E) id[n] = -1;
      l[n] = id[n] >= 0 ? logit(id[n]) : -INFINITY;
      g[n] = id[n] >= 0 ? d_w[static_cast<size_t>(t) * r.top_k + j] : 0.f;
      top = fmaxf(top, l[n]);
    }
    float inv = 1.f;
    if (dense) {
      float sum = 0.f;
      top = -INFINITY;
      for (int e = lane; e < r.E; e += kLanes) top = fmaxf(top, logit(e));
      top = row_max<kLanes>(top);
      for (int e = lane; e < r.E; e += kLanes) {
        const float x = logit(e);
        const float p = x > -INFINITY ? expf(x - top) : 0.f;
        d[e] = p;
        sum += p;
      }
      sum = row_sum<kLanes>(sum);
      inv = sum > 0.f ? 1.f / sum : 0.f;
    } else {
      top = row_max<kLanes>(top);
      for (int e = lane; e < r.E; e += kLanes) d[e] = 0.f;
    }
    float p[2], S = 0.f, dot = 0.f;
    if (r.score == kSigmoid) top = r.renormalise ? fminf(top, 0.f) : 0.f;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      p[n] = l[n] > (r.score == kSigmoid ? kNoSigmoid : -INFINITY) ? score_of(l[n], r.score, top) * inv : 0.f;
      if (RATIO && !(static_cast<double>(l[n]) - most > kNothing)) p[n] = 0.f;
      S += p[n];
      dot += p[n] * g[n];
    }
    S = row_sum<kLanes>(S);
    dot = row_sum<kLanes>(dot);
    const float over = !r.renormalise ? 1.f : S > 0.f ? 1.f / S : 0.f;
    const float mean = r.renormalise ? dot * over : 0.f;
    float across = 0.f;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      g[n] = id[n] >= 0 ? r.scale * over * (g[n] - mean) : 0.f;   // ds of the slot
      if (dense) across += p[n] * g[n];
      else g[n] *= p[n] * (r.score == kSigmoid ? __builtin_amdgcn_rcpf(1.f + expf(l[n])) : 1.f);
    }
    if (dense) {
      across = row_sum<kLanes>(across);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      // p first, as -p sum p ds; the picked ones' p ds follow
      for (int e = lane; e < r.E; e += kLanes) d[e] *= -inv * across;
#pragma unroll
      for (int n = 0; n < 2; ++n) g[n] *= p[n];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    for (int j = 0; j < r.top_k; ++j) {
      const int n = j / kLanes;
      if (lane == j % kLanes && (n ? id[1] : id[0]) >= 0) d[n ? id[1] : id[0]] += n ? g[1] : g[0];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    if (t0 + mine < M) {
      T *out = static_cast<T *>(d_logits) + static_cast<size_t>(t) * r.E;
      struct __attribute__((packed, aligned(sizeof(T)))) Piece {
        T v[16 / sizeof(T)];
      };
      constexpr int P = 16 / sizeof(T);
      for (int e = lane * P; e < r.E; e += kLanes * P) {
        if (e + P <= r.E) {
          Piece o;
#pragma unroll
          for (int i = 0; i < P; ++i) o.v[i] = from_f32<DT>(d[e + i]);
          *reinterpret_cast<Piece *>(out + e) = o;
        } else {
          for (int i = e; i < r.E; ++i) out[i] = from_f32<DT>(d[i]);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

}  // namespace

// tokens of a wavefront times its workgroup's four, and at most so many workgroups
// that the bias is loaded a few times only
static unsigned select_blocks(int M, int tokens) {
  const int per = kWaves * tokens;
  return static_cast<unsigned>(std::min((M + per - 1) / per, 4096));
}

template <int DT>
static void select_go(const MoeSelect &r, const void *logits, int M, const float *bias, int32_t *ids, float *weights,
                      hipStream_t s) {
  const dim3 block(kSelectThreads);
  if (r.groups > kMostGroups)
    hipLaunchKernelGGL(moe_select_exact_kernel<DT>, dim3((M + kWaves - 1) / kWaves), block, 0, s, r, logits, M, bias, ids,
                       weights);
  else if (r.E <= 64)
    hipLaunchKernelGGL((moe_select_kernel<DT, 16, 4>), dim3(select_blocks(M, 4)), block, 0, s, r, logits, M, bias, ids,
                       weights);
  else if (r.E <= 256 && M <= 2048)
    hipLaunchKernelGGL((moe_select_kernel<DT, 64, 4>), dim3(select_blocks(M, 1)), block, 0, s, r, logits, M, bias, ids,
                       weights);
  else if (r.E <= 256)
    hipLaunchKernelGGL((moe_select_kernel<DT, 16, 16>), dim3(select_blocks(M, 4)), block, 0, s, r, logits, M, bias, ids,
                       weights);
  else if (r.E <= 512)
    hipLaunchKernelGGL((moe_select_kernel<DT, 64, 8>), dim3(select_blocks(M, 1)), block, 0, s, r, logits, M, bias, ids,
                       weights);
  else
    hipLaunchKernelGGL((moe_select_kernel<DT, 64, 16>), dim3(select_blocks(M, 1)), block, 0, s, r, logits, M, bias, ids,
                       weights);
}

template <int DT>
static void select_backward_go(const MoeSelect &r, const float *d_w, const void *logits, int M, const int32_t *ids,
                               void *d_logits, hipStream_t s) {
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(select_blocks(M, 4)), dim3(kSelectThreads), 0, s, r, d_w, logits, M, ids, d_logits);
  };
  if (r.score == kSoftmax && r.renormalise) {
    if (r.E <= 64) go(moe_select_backward_kernel<DT, 4, true>);
    else if (r.E <= 256) go(moe_select_backward_kernel<DT, 16, true>);
    else go(moe_select_backward_kernel<DT, 64, true>);
  } else {
    if (r.E <= 64) go(moe_select_backward_kernel<DT, 4, false>);
    else if (r.E <= 256) go(moe_select_backward_kernel<DT, 16, false>);
    else go(moe_select_backward_kernel<DT, 64, false>);
  }
}

hipError_t launch_moe_select(const MoeSelect &r, const void *logits, int dtype, int M, const float *bias, int32_t *ids,
                             float *weights, hipStream_t s) {
  if (dtype == kF16) select_go<kF16>(r, logits, M, bias, ids, weights, s);
  else if (dtype == kBF16) select_go<kBF16>(r, logits, M, bias, ids, weights, s);
  else select_go<kF32>(r, logits, M, bias, ids, weights, s);
  return hipGetLastError();
}

hipError_t launch_moe_select_backward(const MoeSelect &r, const float *d_w, const void *logits, int dtype, int M,
                                      const int32_t *ids, void *d_logits, hipStream_t s) {
  if (dtype == kF16) select_backward_go<kF16>(r, d_w, logits, M, ids, d_logits, s);
  else if (dtype == kBF16) select_backward_go<kBF16>(r, d_w, logits, M, ids, d_logits, s);
  else select_backward_go<kF32>(r, d_w, logits, M, ids, d_logits, s);
  return hipGetLastError();
}

}  // namespace lbq
