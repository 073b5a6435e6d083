// Tokens sorted by expert and back: the counting sort of (token, slot) picks,
// the gather of token rows into sorted order, the weighted combine, and the
// gradients of both. Nothing uses atomics on floating-point data and every sum
// has a fixed order, so repeated calls give identical bits.
#include "device.h"
#include "kernels.h"
#include "mxfp4.h"

#include <algorithm>

namespace lbq {

namespace {

using namespace mxfp4;

// ------------------------------------------------------------------ sort

constexpr int kSortWaves = 16, kSortThreads = 64 * kSortWaves;
constexpr int kMaxBlocks = 64;

// Picks per workgroup: all of up to 4096; else at least 2048 in whole
// 1024-chunks, at most kMaxBlocks workgroups (each reads every other's counts).
// 131072 picks of 256 experts: 64 workgroups 15 us, 8 workgroups 36.
int sort_chunk(int n) {
  if (n <= 4096) return std::max(1, (n + kSortThreads - 1) / kSortThreads) * kSortThreads;
  const int per = (n + kMaxBlocks - 1) / kMaxBlocks;
  return std::max(2048, (per + kSortThreads - 1) / kSortThreads * kSortThreads);
}

__device__ __forceinline__ int expert_of(const int32_t *ids, int a, int end, int E) {
  if (a >= end) return -1;
  const int e = ids[a];
  return e >= 0 && e < E ? e : -1;
}

// Counts of one workgroup's chunk (integer sums: the order does not matter).
__global__ void __launch_bounds__(kSortThreads) moe_hist_kernel(const int32_t *__restrict__ ids, int n, int E,
                                                                int chunk, int32_t *__restrict__ hist) {
  __shared__ int32_t cnt[kMoeMaxExperts];
  for (int i = threadIdx.x; i < E; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  const int lo = blockIdx.x * chunk, hi = min(n, lo + chunk);
  for (int a = lo + threadIdx.x; a < hi; a += kSortThreads) {
    const int e = expert_of(ids, a, hi, E);
    if (e >= 0) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < E; i += kSortThreads) hist[static_cast<size_t>(blockIdx.x) * E + i] = cnt[i];
}

// Places one workgroup's chunk. Wave w owns the w-th sixteenth of the chunk and
// walks it in order, 64 picks at a time: a pick's place is its expert's start
// plus the picks of that expert before it (other workgroups' from hist, other
// waves' from the LDS counts, its own wave's earlier ones from the running
// count, and among the 64 by a ballot over the bits of the expert number).
// hist is null where one workgroup holds every pick.
__global__ void __launch_bounds__(kSortThreads) moe_place_kernel(const int32_t *__restrict__ ids, int n, int E,
                                                                 int chunk, const int32_t *__restrict__ hist,
                                                                 int32_t *__restrict__ counts,
                                                                 int32_t *__restrict__ offsets,
                                                                 int32_t *__restrict__ perm,
                                                                 int32_t *__restrict__ pos) {
  __shared__ int32_t s_cnt[kSortWaves * kMoeMaxExperts];   // per (wave, expert): count, then the running place
  __shared__ int32_t s_wave[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lo = blockIdx.x * chunk, hi = min(n, lo + chunk);
  const int per_wave = (chunk + kSortWaves - 1) / kSortWaves;
  const int w_lo = min(hi, lo + wave * per_wave), w_hi = min(hi, w_lo + per_wave);
  for (int i = tid; i < kSortWaves * E; i += kSortThreads) s_cnt[i] = 0;
  __syncthreads();
  for (int a = w_lo + lane; a < w_hi; a += 64) {
    const int e = expert_of(ids, a, w_hi, E);
    if (e >= 0) atomicAdd(&s_cnt[wave * E + e], 1);
  }
  __syncthreads();
  // thread e: the expert's picks in all, and those before this workgroup
  int total = 0, before = 0;
  if (tid < E) {
    if (hist) {
      const int blocks = gridDim.x, mine = blockIdx.x;
      for (int b0 = 0; b0 < blocks; b0 += 16) {
        int c[16];   // sixteen loads under way
#pragma unroll
        for (int i = 0; i < 16; ++i) c[i] = b0 + i < blocks ? hist[(b0 + i) * E + tid] : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          total += c[i];
          before += b0 + i < mine ? c[i] : 0;
        }
      }
    } else {
      for (int w = 0; w < kSortWaves; ++w) total += s_cnt[w * E + tid];
    }
  }
  // exclusive scan of the totals over the experts (one per thread)
  int incl = total;
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 63) s_wave[wave] = incl;
  __syncthreads();
  int base = 0, all = 0;
  for (int w = 0; w < kSortWaves; ++w) {
    if (w < wave) base += s_wave[w];
    all += s_wave[w];
  }
  const int start = base + incl - total;
  if (tid < E) {
    int run = start + before;
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = s_cnt[w * E + tid];
      s_cnt[w * E + tid] = run;
      run += c;
    }
    if (blockIdx.x == 0) {
      counts[tid] = total;
      offsets[tid] = start;
      if (tid == 0) offsets[E] = all;
    }
  }
  __syncthreads();
  const int bits = 32 - __builtin_clz(max(E - 1, 1));
  for (int a0 = w_lo; a0 < w_hi; a0 += 64) {
    const int a = a0 + lane;
    const int e = expert_of(ids, a, w_hi, E);
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t bal = __ballot((e >> b) & 1);
      same &= ((e >> b) & 1) ? bal : ~bal;
    }
    if (e >= 0) {
      const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
      const int p = s_cnt[wave * E + e] + rank;
      // the last of the equal lanes moves the running place on (the reads
      // above are done: a wave's LDS operations complete in order)
      __builtin_amdgcn_wave_barrier();
      if ((same >> lane) == 1) s_cnt[wave * E + e] = p + 1;
      perm[p] = a;
      pos[a] = p;
    } else if (a < w_hi) {
      pos[a] = -1;
    }
    __builtin_amdgcn_wave_barrier();
  }
  // places behind the last pick
  for (int a = lo + tid; a < hi; a += kSortThreads)
    if (a >= all) perm[a] = -1;
}

// ------------------------------------------------------------------ rows

// V values of a row at once: eight (16-byte vectors) where rows are whole
// vectors, else one.
template <int DT, int V>
struct Row {
  using T = typename Elem<DT>::type;
  T v[V];
  static __device__ __forceinline__ Row load(const void *p, size_t at) {
    Row r;
    if constexpr (V == 1) {
      r.v[0] = static_cast<const T *>(p)[at];
    } else {
      constexpr int kVecs = V * sizeof(T) / 16;
      uint4 *q = reinterpret_cast<uint4 *>(r.v);
#pragma unroll
      for (int i = 0; i < kVecs; ++i) q[i] = reinterpret_cast<const uint4 *>(static_cast<const T *>(p) + at)[i];
    }
    return r;
  }
  // PAST: past the caches
  template <bool PAST = false>
  __device__ __forceinline__ void store(void *p, size_t at) const {
    if constexpr (V == 1) {
      static_cast<T *>(p)[at] = v[0];
    } else {
      typedef uint32_t vec_t __attribute__((ext_vector_type(4)));
      constexpr int kVecs = V * sizeof(T) / 16;
      const vec_t *q = reinterpret_cast<const vec_t *>(v);
      vec_t *o = reinterpret_cast<vec_t *>(static_cast<T *>(p) + at);
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        if constexpr (PAST) __builtin_nontemporal_store(q[i], o + i);
        else o[i] = q[i];
      }
    }
  }
};

constexpr int kRowThreads = 256;

// out[pos[t][j]] = x[t]: each token row is read once and written top_k times.
// PAST: a list larger than the memory-side cache goes past it. 131072 rows of
// 4 KB: the gather itself takes 117 instead of 87 us, what reads such a list
// next 113 instead of 150 (it need not wait for the cache to be written back).
template <int DT, int V, bool PAST>
__global__ void __launch_bounds__(kRowThreads) moe_gather_kernel(const void *__restrict__ x, int M, int H, int T,
                                                                 const int32_t *__restrict__ pos, int top_k,
                                                                 void *__restrict__ out) {
  const int t = blockIdx.x;
  for (int c = (blockIdx.y * kRowThreads + threadIdx.x) * V; c < H; c += gridDim.y * kRowThreads * V) {
    const auto r = Row<DT, V>::load(x, static_cast<size_t>(t) * H + c);
    for (int j = 0; j < top_k; ++j) {
      const int p = pos[static_cast<size_t>(t) * top_k + j];
      if (p >= 0 && p < T) r.template store<PAST>(out, static_cast<size_t>(p) * H + c);
    }
  }
}

// Picks of one token at a time: their rows are all under way before the first
// is used.
constexpr int kCombinePicks = 8, kBackwardPicks = 2;

// The places of picks j0 .. j0 + N - 1 of token t (one token per
// workgroup: scalar loads). A pick past the last, or without a place in [0, T),
// is not there; its row number is one that can be read all the same.
template <int N>
struct Picks {
  int row[N];
  bool there[N];
  __device__ __forceinline__ Picks(const int32_t *pos, int t, int top_k, int j0, int T) {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int p = pos[static_cast<size_t>(t) * top_k + min(j0 + u, top_k - 1)];
      there[u] = j0 + u < top_k && p >= 0 && p < T;
      row[u] = there[u] ? p : 0;
    }
  }
};

// y[t] = sum_j w[t][j] o[pos[t][j]] in fp32, slot order; w null: all ones.
// Bound: HBM. 16384 tokens, 8 picks, rows of 4 KB (0.58 GB): 116 to 135 us, 5.0
// to 4.3 TB/s (155 with one row under way at a time).
template <int DT, int V>
__global__ void __launch_bounds__(kRowThreads) moe_combine_kernel(const void *__restrict__ o, int T, int H,
                                                                  const int32_t *__restrict__ pos,
                                                                  const float *__restrict__ w, int top_k,
                                                                  void *__restrict__ y) {
  constexpr int kPicks = kCombinePicks;
  const int t = blockIdx.x;
  for (int c = (blockIdx.y * kRowThreads + threadIdx.x) * V; c < H; c += gridDim.y * kRowThreads * V) {
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    for (int j0 = 0; j0 < (T > 0 ? top_k : 0); j0 += kPicks) {
      const Picks<kPicks> p(pos, t, top_k, j0, T);
      Row<DT, V> r[kPicks];
#pragma unroll
      for (int u = 0; u < kPicks; ++u)
        if (j0 + u < top_k) r[u] = Row<DT, V>::load(o, static_cast<size_t>(p.row[u]) * H + c);
#pragma unroll
      for (int u = 0; u < kPicks; ++u) {
        if (!p.there[u]) continue;
        const float wj = w ? w[static_cast<size_t>(t) * top_k + j0 + u] : 1.f;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(wj, to_f32<DT>(r[u].v[i]), acc[i]);
      }
    }
    Row<DT, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = from_f32<DT>(acc[i]);
    r.store(y, static_cast<size_t>(t) * H + c);
  }
}

// d_o[pos[t][j]] = w[t][j] dy[t];  d_w[t][j] = <dy[t], o[pos[t][j]]>, summed per
// thread over its columns, then over the wave, then over the waves in order.
// d_o may be o (each value is read before its place is written).
// Bound: HBM. 16384 tokens, 8 picks, rows of 4 KB (1.15 GB): 210 us, 5.5 TB/s.
// Rows under way, 1, 2 or 4: 1024 tokens 12.7, 14.1, 15.6 us; 32 tokens 7.2, 7.2,
// 6.5; 8192 tokens, 4 picks, fp32 rows of 16 KB 256, 250, 260.
template <int DT, int V>
__global__ void __launch_bounds__(kRowThreads) moe_combine_backward_kernel(
    const void *__restrict__ dy, const void *o, int T, int H, const int32_t *__restrict__ pos,
    const float *__restrict__ w, int top_k, void *d_o, float *__restrict__ d_w) {
  constexpr int kWaves = kRowThreads / 64, kPicks = kBackwardPicks;
  __shared__ float part[kWaves][kPicks];
  const int t = blockIdx.x;
  for (int j0 = 0; j0 < top_k; j0 += kPicks) {
    const Picks<kPicks> p(pos, t, top_k, j0, T);
    float dot[kPicks];
#pragma unroll
    for (int u = 0; u < kPicks; ++u) dot[u] = 0.f;
    for (int c = threadIdx.x * V; c < (T > 0 ? H : 0); c += kRowThreads * V) {
      const auto g = Row<DT, V>::load(dy, static_cast<size_t>(t) * H + c);
      Row<DT, V> r[kPicks];
#pragma unroll
      for (int u = 0; u < kPicks; ++u)
        if (j0 + u < top_k) r[u] = Row<DT, V>::load(o, static_cast<size_t>(p.row[u]) * H + c);
#pragma unroll
      for (int u = 0; u < kPicks; ++u) {
        if (!p.there[u]) continue;
        const float wj = w[static_cast<size_t>(t) * top_k + j0 + u];
        Row<DT, V> d;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float gi = to_f32<DT>(g.v[i]);
          dot[u] = fmaf(gi, to_f32<DT>(r[u].v[i]), dot[u]);
          d.v[i] = from_f32<DT>(wj * gi);
        }
        d.store(d_o, static_cast<size_t>(p.row[u]) * H + c);
      }
    }
#pragma unroll
    for (int u = 0; u < kPicks; ++u) {
      for (int x = 32; x > 0; x /= 2) dot[u] += __shfl_xor(dot[u], x);
      if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6][u] = dot[u];
    }
    __syncthreads();
    if (threadIdx.x < kPicks && j0 + static_cast<int>(threadIdx.x) < top_k) {
      float sum = 0.f;
      for (int i = 0; i < kWaves; ++i) sum += part[i][threadIdx.x];
      d_w[static_cast<size_t>(t) * top_k + j0 + threadIdx.x] = sum;
    }
    __syncthreads();
  }
}

template <int DT, int V>
constexpr auto gather_past = moe_gather_kernel<DT, V, true>;
template <int DT, int V>
constexpr auto gather_kept = moe_gather_kernel<DT, V, false>;

unsigned chunks(int H, int v) {
  return static_cast<unsigned>(std::min((H + kRowThreads * v - 1) / (kRowThreads * v), 64));
}

}  // namespace

size_t moe_sort_ws_bytes(int n, int E) {
  const int chunk = sort_chunk(n);
  return n <= chunk ? 0 : static_cast<size_t>((n + chunk - 1) / chunk) * E * 4;
}

hipError_t launch_moe_sort(const int32_t *ids, int n, int E, int32_t *counts, int32_t *offsets, int32_t *perm,
                           int32_t *pos, void *ws, hipStream_t s) {
  const int chunk = sort_chunk(n);
  const int blocks = std::max(1, (n + chunk - 1) / chunk);
  int32_t *hist = blocks > 1 ? static_cast<int32_t *>(ws) : nullptr;
  if (hist) hipLaunchKernelGGL(moe_hist_kernel, dim3(blocks), dim3(kSortThreads), 0, s, ids, n, E, chunk, hist);
  hipLaunchKernelGGL(moe_place_kernel, dim3(blocks), dim3(kSortThreads), 0, s, ids, n, E, chunk, hist, counts, offsets,
                     perm, pos);
  return hipGetLastError();
}

// eight values a lane where every row starts on a 16-byte boundary, else one: 16384
// tokens, 8 picks, bf16 rows of 2048 and of 2047 or 2044 values: gather 104 and 253
// us, combine 121 and 183, its gradient 230 and 398
#define LBQ_ROWS(KERNEL, GRIDY, ...)                                                                        \
  do {                                                                                                      \
    const bool vec = H % 8 == 0;                                                                            \
    const dim3 grid(static_cast<unsigned>(M), GRIDY ? chunks(H, vec ? 8 : 1) : 1), block(kRowThreads);      \
    if (dtype == kF16 && vec) hipLaunchKernelGGL((KERNEL<kF16, 8>), grid, block, 0, s, __VA_ARGS__);        \
    else if (dtype == kF16) hipLaunchKernelGGL((KERNEL<kF16, 1>), grid, block, 0, s, __VA_ARGS__);          \
    else if (dtype == kBF16 && vec) hipLaunchKernelGGL((KERNEL<kBF16, 8>), grid, block, 0, s, __VA_ARGS__); \
    else if (dtype == kBF16) hipLaunchKernelGGL((KERNEL<kBF16, 1>), grid, block, 0, s, __VA_ARGS__);        \
    else if (vec) hipLaunchKernelGGL((KERNEL<kF32, 8>), grid, block, 0, s, __VA_ARGS__);                    \
    else hipLaunchKernelGGL((KERNEL<kF32, 1>), grid, block, 0, s, __VA_ARGS__);                             \
  } while (0)

hipError_t launch_moe_gather(const void *x, int dtype, int M, int H, int T, const int32_t *pos, int top_k, void *out,
                             hipStream_t s) {
  constexpr size_t kMemorySideCache = size_t{256} << 20;
  const size_t bytes = static_cast<size_t>(M) * top_k * H * (dtype == kF32 ? 4 : 2);
  if (bytes > kMemorySideCache) LBQ_ROWS(gather_past, true, x, M, H, T, pos, top_k, out);
  else LBQ_ROWS(gather_kept, true, x, M, H, T, pos, top_k, out);
  return hipGetLastError();
}

hipError_t launch_moe_combine(const void *o, int dtype, int T, int H, const int32_t *pos, const float *weights, int M,
                              int top_k, void *y, hipStream_t s) {
  LBQ_ROWS(moe_combine_kernel, true, o, T, H, pos, weights, top_k, y);
  return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const void *dy, const void *o, int dtype, int T, int H, const int32_t *pos,
                                       const float *weights, int M, int top_k, void *d_o, float *d_w, hipStream_t s) {
  LBQ_ROWS(moe_combine_backward_kernel, false, dy, o, T, H, pos, weights, top_k, d_o, d_w);
  return hipGetLastError();
}

}  // namespace lbq
