// The C ABI of the expert selection and the low-rank adapters (include/lbq.h):
// argument checks, workspace layout, and kernel launches on the caller's
// stream. No allocation, no global state.
#include <hip/hip_runtime.h>

#include "../../include/lbq.h"
#include "kernels.h"

using namespace lbq;

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxPicks = 1 << 24, kMaxCols = 1 << 24;

inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline lbq_status hip_status(hipError_t e) { return e == hipSuccess ? LBQ_OK : LBQ_ERR_HIP; }

lbq_status check_router(const lbq_router *r, int32_t dtype, int32_t M) {
  if (!r) return LBQ_ERR_NULL;
  if (r->E < 1 || r->E > kMoeMaxExperts || r->top_k < 1 || r->top_k > r->E || r->top_k > kMoeMaxTopK)
    return LBQ_ERR_SHAPE;
  if (r->groups < 1 || r->E % r->groups != 0 || r->top_groups < 1 || r->top_groups > r->groups ||
      r->group_picks < 1 || r->group_picks > 2 || r->top_k > r->E / r->groups * r->top_groups)
    return LBQ_ERR_SHAPE;
  if (M < 0 || static_cast<int64_t>(M) * r->top_k > kMaxPicks) return LBQ_ERR_SHAPE;
  if (r->score != LBQ_SCORE_SOFTMAX && r->score != LBQ_SCORE_SIGMOID) return LBQ_ERR_FORMAT;
  return dtype >= LBQ_F16 && dtype <= LBQ_F32 ? LBQ_OK : LBQ_ERR_FORMAT;
}

MoeSelect select_args(const lbq_router *r) {
  return {r->E, r->top_k, r->score, r->groups, r->top_groups, r->group_picks, r->renormalise != 0, r->scale};
}

lbq_status check_adapters(const lbq_adapters *ad, int32_t M) {
  if (!ad) return LBQ_ERR_NULL;
  if (ad->L < 1 || ad->L > kMoeMaxExperts || ad->K < 1 || ad->K > kMaxCols || ad->K % 128 != 0 || ad->N < 1 ||
      ad->N > kMaxCols || ad->r < 1 || ad->r > kAdapterMaxRank)
    return LBQ_ERR_SHAPE;
  if (M < 0 || M > kMoeMaxAssignments) return LBQ_ERR_SHAPE;
  if (ad->dtype != LBQ_F16 && ad->dtype != LBQ_BF16) return LBQ_ERR_FORMAT;
  if (!ad->a || !ad->b || !ad->scales) return LBQ_ERR_NULL;
  return aligned(ad->a, 16) && aligned(ad->b, 16) && aligned(ad->scales, 4) ? LBQ_OK : LBQ_ERR_ALIGN;
}

AdapterArgs adapter_args(const lbq_adapters *ad, int32_t M) {
  AdapterArgs g{};
  g.L = ad->L;
  g.K = ad->K;
  g.N = ad->N;
  g.r = ad->r;
  g.M = M;
  g.dtype = ad->dtype;
  g.a = ad->a;
  g.b = ad->b;
  g.scales = ad->scales;
  return g;
}

// The sort's results where the caller gives none, then the kernels' scratch.
struct AdapterLayout {
  size_t counts = 0, offsets = 0, perm = 0, pos = 0, sort = 0, scratch = 0, total = 0;
};
AdapterLayout adapter_layout(const AdapterArgs &g, bool sorts, bool backward) {
  AdapterLayout l;
  if (sorts) {
    l.offsets = round_up(4 * static_cast<size_t>(g.L), kAlign);
    l.perm = l.offsets + round_up(4 * (static_cast<size_t>(g.L) + 1), kAlign);
    l.pos = l.perm + round_up(4 * static_cast<size_t>(g.M), kAlign);
    l.sort = l.pos + round_up(4 * static_cast<size_t>(g.M), kAlign);
    l.scratch = l.sort + round_up(moe_sort_ws_bytes(g.M, g.L), kAlign);
  }
  l.total = l.scratch + (backward ? adapters_backward_ws_bytes(g) : adapters_forward_ws_bytes(g));
  return l;
}

// Whether a call makes the order itself; the query and the calls ask here.
bool makes_order(const AdapterArgs &g, bool given, bool backward) {
  return !given && (backward || adapters_forward_by_list(g));
}

lbq_status workspace(const lbq_adapters *ad, int32_t M, int32_t sorted, bool backward, size_t *bytes) {
  if (!bytes) return LBQ_ERR_NULL;
  const lbq_status st = check_adapters(ad, M);
  if (st != LBQ_OK) return st;
  const AdapterArgs g = adapter_args(ad, M);
  *bytes = adapter_layout(g, makes_order(g, sorted != 0, backward), backward).total;
  return LBQ_OK;
}

// The sorted order the caller gave, or one made in the workspace.
lbq_status order(AdapterArgs &g, const int32_t *offsets, const int32_t *perm, bool sorts, const AdapterLayout &l,
                 uint8_t *base, hipStream_t s) {
  g.offsets = offsets;
  g.perm = perm;
  g.scratch = base ? base + l.scratch : nullptr;
  if (!sorts) return LBQ_OK;
  auto at = [&](size_t o) { return reinterpret_cast<int32_t *>(base + o); };
  g.offsets = at(l.offsets);
  g.perm = at(l.perm);
  return hip_status(launch_moe_sort(g.ids, g.M, g.L, at(l.counts), at(l.offsets), at(l.perm), at(l.pos),
                                    base + l.sort, s));
}

}  // namespace

extern "C" {

lbq_status lbq_moe_select(const lbq_router *r, const void *logits, int32_t dtype, int32_t M, const float *bias,
                          int32_t *ids, float *weights, void *stream) {
  const lbq_status st = check_router(r, dtype, M);
  if (st != LBQ_OK) return st;
  if (M == 0) return LBQ_OK;
  if (!logits || !ids || !weights) return LBQ_ERR_NULL;
  if (!aligned(logits, 16) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4)) return LBQ_ERR_ALIGN;
  return hip_status(launch_moe_select(select_args(r), logits, dtype, M, bias, ids, weights,
                                      static_cast<hipStream_t>(stream)));
}

lbq_status lbq_moe_select_backward(const lbq_router *r, const float *d_weights, const void *logits, int32_t dtype,
                                   const int32_t *ids, int32_t M, void *d_logits, void *stream) {
  const lbq_status st = check_router(r, dtype, M);
  if (st != LBQ_OK) return st;
  if (M == 0) return LBQ_OK;
  if (!d_weights || !logits || !ids || !d_logits) return LBQ_ERR_NULL;
  if (!aligned(logits, 16) || !aligned(d_logits, 16) || !aligned(ids, 4) || !aligned(d_weights, 4))
    return LBQ_ERR_ALIGN;
  return hip_status(launch_moe_select_backward(select_args(r), d_weights, logits, dtype, M, ids, d_logits,
                                               static_cast<hipStream_t>(stream)));
}

lbq_status lbq_adapters_workspace(const lbq_adapters *ad, int32_t M, int32_t sorted, size_t *bytes) {
  return workspace(ad, M, sorted, false, bytes);
}

lbq_status lbq_adapters_backward_workspace(const lbq_adapters *ad, int32_t M, int32_t sorted, size_t *bytes) {
  return workspace(ad, M, sorted, true, bytes);
}

lbq_status lbq_adapters_forward(const lbq_adapters *ad, const void *x, int32_t M, const int32_t *ids,
                                const int32_t *offsets, const int32_t *perm, const void *base, void *y, float *h,
                                void *ws, size_t ws_bytes, void *stream) {
  lbq_status st = check_adapters(ad, M);
  if (st != LBQ_OK) return st;
  if (M == 0) return LBQ_OK;
  if (!x || !ids || !y || (!offsets) != (!perm)) return LBQ_ERR_NULL;
  if (!aligned(x, 16) || !aligned(base, 16) || !aligned(y, 16) || !aligned(h, 4) || !aligned(ids, 4) ||
      !aligned(offsets, 4) || !aligned(perm, 4) || !aligned(ws, 16))
    return LBQ_ERR_ALIGN;
  AdapterArgs g = adapter_args(ad, M);
  const bool sorts = makes_order(g, offsets != nullptr, false);
  const AdapterLayout l = adapter_layout(g, sorts, false);
  if (l.total > 0 && !ws) return LBQ_ERR_NULL;
  if (ws_bytes < l.total) return LBQ_ERR_WORKSPACE;
  g.x = x;
  g.ids = ids;
  g.base = base;
  g.y = y;
  g.h = h;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  st = order(g, offsets, perm, sorts, l, static_cast<uint8_t *>(ws), s);
  return st != LBQ_OK ? st : hip_status(launch_adapters_forward(g, s));
}

lbq_status lbq_adapters_backward(const lbq_adapters *ad, const void *dy, const void *x, const float *h, int32_t M,
                                 const int32_t *ids, const int32_t *offsets, const int32_t *perm, const void *base,
                                 void *dx, float *d_a, float *d_b, void *ws, size_t ws_bytes, void *stream) {
  lbq_status st = check_adapters(ad, M);
  if (st != LBQ_OK) return st;
  if (!d_a || !d_b || (M > 0 && (!dy || !x || !h || !ids || !dx || (!offsets) != (!perm)))) return LBQ_ERR_NULL;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(h, 4) || !aligned(ids, 4) || !aligned(offsets, 4) ||
      !aligned(perm, 4) || !aligned(base, 16) || !aligned(dx, 16) || !aligned(d_a, 16) || !aligned(d_b, 16) ||
      !aligned(ws, 16))
    return LBQ_ERR_ALIGN;
  AdapterArgs g = adapter_args(ad, M);
  const bool sorts = makes_order(g, offsets != nullptr, true);   // (M = 0: offsets alone, of whatever values)
  const AdapterLayout l = adapter_layout(g, sorts, true);
  if (l.total > 0 && !ws) return LBQ_ERR_NULL;
  if (ws_bytes < l.total) return LBQ_ERR_WORKSPACE;
  g.dy = dy;
  g.x = x;
  g.h = const_cast<float *>(h);
  g.ids = ids;
  g.base = base;
  g.y = dx;
  g.d_a = d_a;
  g.d_b = d_b;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  st = order(g, offsets, perm, sorts, l, static_cast<uint8_t *>(ws), s);
  return st != LBQ_OK ? st : hip_status(launch_adapters_backward(g, s));
}

}  // extern "C"
