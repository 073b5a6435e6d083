// The C ABI of the MXFP4 tensors and the expert dispatch (include/lbq.h):
// argument checks, workspace layout, and kernel launches on the caller's
// stream. No allocation, no global state.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../include/lbq.h"
#include "kernels.h"

using namespace lbq;

namespace {

constexpr size_t kAlign = 256;

inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline lbq_status hip_status(hipError_t e) { return e == hipSuccess ? LBQ_OK : LBQ_ERR_HIP; }

inline bool value_type(int32_t dtype) { return dtype >= LBQ_F16 && dtype <= LBQ_F32; }
inline bool half_type(int32_t dtype) { return dtype == LBQ_F16 || dtype == LBQ_BF16; }

// (row numbers and their roundings up to whole tiles stay 32-bit, and so do the
// offsets within 256 rows)
constexpr int64_t kMaxRows = 1 << 30, kMaxCols = 1 << 24;

bool mx_shape(int64_t rows, int64_t cols) {
  return rows >= 0 && rows <= kMaxRows && cols > 0 && cols <= kMaxCols && cols % 128 == 0 &&
         rows * (cols / 128) < (1ll << 31);
}
size_t code_bytes(int64_t rows, int64_t cols) { return static_cast<size_t>(rows) * (cols / 2); }
size_t scale_bytes(int64_t rows, int64_t cols) { return static_cast<size_t>(rows) * (cols / 32); }

lbq_status check_mx(const lbq_mx *t) {
  if (!t) return LBQ_ERR_NULL;
  if (!mx_shape(t->rows, t->cols)) return LBQ_ERR_SHAPE;
  if (t->rows > 0 && (!t->codes || !t->scales)) return LBQ_ERR_NULL;
  if (!aligned(t->codes, 16) || !aligned(t->scales, 16)) return LBQ_ERR_ALIGN;
  return LBQ_OK;
}

lbq_status check_matmul(const lbq_mx *a, const lbq_mx *b) {
  lbq_status st = check_mx(a);
  if (st == LBQ_OK) st = check_mx(b);
  if (st != LBQ_OK) return st;
  return a->cols == b->cols ? LBQ_OK : LBQ_ERR_SHAPE;
}

MxGemm dense(int M, const lbq_mx *b, void *y, int32_t dtype) {
  MxGemm g{};
  g.b_codes = b->codes;
  g.b_scales = b->scales;
  g.y = y;
  g.dtype = dtype;
  g.a_rows = g.M = M;
  g.N = b->rows;
  g.K = b->cols;
  g.top_k = 1;
  return g;
}

// Rows of a tile on the streaming kernel, 0: the tile kernel. Grouped: where 16
// rows hold the average expert's and half as many again (256 experts of 2048 x
// 2048, 4 rows: 105 us, the tile kernel 115; 8 rows: 115, 119; 12 rows: 141, 125).
int stream_rows(const MxGemm &g) {
  const long rows = g.E > 0 ? (3l * g.M + 2 * g.E - 1) / (2 * g.E) : g.M;
  for (int t = 16; t <= (g.E > 0 ? 16 : 64); t *= 2)
    if (rows <= t && mx_stream_supported(t, g.K)) return t;
  return 0;
}

// The streaming kernel quantizes the activations itself where every workgroup
// doing so costs about as much as a launch, or less; that work is a workgroup's
// tokens times K, for an expert's rows their average. Itself against with a launch
// before it, us a call in a graph (one by one), and the work:
//   8 x 4096 -> 4096     6.2 (6.5)     7.0 (9.2)     2^15
//   16 x 4096 -> 4096    7.9 (8.1)     7.3 (9.2)     2^16
//   4 x 14336 -> 4096    14.3 (14.1)   14.8 (14.4)   0.9 2^16
//   8 x 8192 -> 4096     10.8 (10.7)   10.1 (10.1)   2^16; -> 8192 13.6, 13.7
//   8 x 14336 -> 4096    16.9 (16.7)   16.2 (15.8)   1.8 2^16
//   8 x 17408 -> 4096    17.7 (17.7)   16.3 (16.3)   2.1 2^16
//   16 x 8192 -> 4096    14.2 (13.9)   10.9 (10.7)   2^17
//   32 x 2048 -> 4096    7.2 (7.1)     6.7 (9.4)     2^16
//   33 x 1024 -> 4096    9.2 (8.8)     7.2 (9.4)     2^15
//   64 x 512 -> 4096     10.5 (10.6)   7.2 (8.9)     2^15
//   256 experts of 2048 x 2048, 8 rows each   141.3   144.7   2^14
//   16 of 4096 x 4096, 2.5 rows               34.0    35.3    0.6 2^14
//   16 of 4096 x 4096, 10 rows                39.6    39.0    1.3 2^15
//   16 of 4096 x 8192, 8 rows                 63.8    60.6    2^16
//   8 of 4096 x 14336, 4 rows                 83.6    77.6    0.9 2^16
bool stream_quantizes(const MxGemm &g) {
  if (stream_rows(g) == 0) return false;
  const long work = static_cast<long>(g.M) * g.K;
  return g.E > 0 ? work < static_cast<long>(g.E) << 15 : g.M <= 32 && work <= 1 << 16;
}

size_t scratch_bytes(const MxGemm &g) { return stream_rows(g) > 0 ? 0 : mx_gemm_scratch_bytes(g); }

// The quantized activations of M rows (none where the product takes x itself),
// then the product's scratch.
struct LinearLayout {
  size_t scales = 0, scratch = 0, total = 0;
};
LinearLayout linear_layout(int M, int K, const MxGemm &g) {
  LinearLayout l;
  if (stream_quantizes(g)) return l;
  l.scales = round_up(code_bytes(M, K), kAlign);
  l.scratch = l.scales + round_up(scale_bytes(M, K), kAlign);
  l.total = l.scratch + scratch_bytes(g);
  return l;
}

hipError_t launch_product(const MxGemm &g, hipStream_t s) {
  const int rows = stream_rows(g);
  return rows > 0 ? launch_mx_stream(g, rows, s) : launch_mx_gemm(g, s);
}

// Q(x) into the workspace, unless the product takes x itself; then the product.
lbq_status quantize_and_multiply(MxGemm g, const void *x, void *ws, const LinearLayout &l, hipStream_t s) {
  if (stream_quantizes(g)) {
    g.x = x;
    return hip_status(launch_product(g, s));
  }
  uint8_t *base = static_cast<uint8_t *>(ws);
  if (launch_mx_quantize(x, g.dtype, g.a_rows, g.K, base, base + l.scales, s) != hipSuccess) return LBQ_ERR_HIP;
  g.a_codes = base;
  g.a_scales = base + l.scales;
  g.scratch = base + l.scratch;
  return hip_status(launch_product(g, s));
}

lbq_status check_grouped(const lbq_mx *w, int32_t E, int32_t M, int32_t T) {
  const lbq_status st = check_mx(w);
  if (st != LBQ_OK) return st;
  if (E < 1 || E > kMoeMaxExperts || w->rows % E != 0 || T < 0 || T > kMaxRows) return LBQ_ERR_SHAPE;
  if (!mx_shape(M, w->cols)) return LBQ_ERR_SHAPE;
  // the quantized rows, taken in any order, at 32-bit offsets
  if (code_bytes(M, w->cols) >= 1ull << 32) return LBQ_ERR_SHAPE;
  return LBQ_OK;
}

MxGemm grouped(const lbq_mx *w, int32_t E, int32_t M, int32_t T) {
  MxGemm g = dense(T, w, nullptr, LBQ_F16);
  g.a_rows = M;
  g.N = w->rows / E;
  g.E = E;
  return g;
}

lbq_status check_picks(int32_t M, int32_t top_k) {
  if (M < 0 || top_k < 1 || top_k > kMoeMaxTopK) return LBQ_ERR_SHAPE;
  return static_cast<long>(M) * top_k <= kMoeMaxAssignments ? LBQ_OK : LBQ_ERR_SHAPE;
}

lbq_status check_rows(int32_t dtype, int32_t M, int32_t top_k, int32_t T, int32_t H) {
  const lbq_status st = check_picks(M, top_k);
  if (st != LBQ_OK) return st;
  if (T < 0 || H < 1 || H > kMaxRows) return LBQ_ERR_SHAPE;
  return value_type(dtype) ? LBQ_OK : LBQ_ERR_FORMAT;
}

}  // namespace

extern "C" {

lbq_status lbq_mx_bytes(int32_t rows, int32_t cols, size_t *code_bytes_out, size_t *scale_bytes_out) {
  if (!code_bytes_out || !scale_bytes_out) return LBQ_ERR_NULL;
  if (!mx_shape(rows, cols)) return LBQ_ERR_SHAPE;
  *code_bytes_out = code_bytes(rows, cols);
  *scale_bytes_out = scale_bytes(rows, cols);
  return LBQ_OK;
}

lbq_status lbq_mx_quantize(const void *x, int32_t dtype, int32_t rows, int32_t cols, void *codes, void *scales,
                           void *stream) {
  if (!mx_shape(rows, cols)) return LBQ_ERR_SHAPE;
  if (!value_type(dtype)) return LBQ_ERR_FORMAT;
  if (rows == 0) return LBQ_OK;
  if (!x || !codes || !scales) return LBQ_ERR_NULL;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 16)) return LBQ_ERR_ALIGN;
  return hip_status(launch_mx_quantize(x, dtype, rows, cols, codes, scales, static_cast<hipStream_t>(stream)));
}

lbq_status lbq_mx_quantize_t(const void *x, int32_t dtype, int32_t rows, int32_t cols, void *codes, void *scales,
                             void *stream) {
  if (rows < 0 || cols < 1) return LBQ_ERR_SHAPE;
  const int64_t padded = (static_cast<int64_t>(rows) + 127) / 128 * 128;
  // the transposed tensor's columns are an int32, its row groups a grid dimension,
  // and so are 64 of its rows, of 256 threads
  if (padded > INT32_MAX || padded / 128 > 65535 || cols > kMaxRows - 64 ||
      (rows > 0 && !mx_shape(cols, padded)))
    return LBQ_ERR_SHAPE;
  if (!value_type(dtype)) return LBQ_ERR_FORMAT;
  if (rows == 0) return LBQ_OK;
  if (!x || !codes || !scales) return LBQ_ERR_NULL;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 16)) return LBQ_ERR_ALIGN;
  return hip_status(launch_mx_quantize_t(x, dtype, rows, cols, codes, scales, static_cast<hipStream_t>(stream)));
}

lbq_status lbq_mx_dequantize(const lbq_mx *t, void *x, int32_t dtype, void *stream) {
  const lbq_status st = check_mx(t);
  if (st != LBQ_OK) return st;
  if (!value_type(dtype)) return LBQ_ERR_FORMAT;
  if (t->rows == 0) return LBQ_OK;
  if (!x) return LBQ_ERR_NULL;
  if (!aligned(x, 16)) return LBQ_ERR_ALIGN;
  return hip_status(
      launch_mx_dequantize(t->codes, t->scales, t->rows, t->cols, x, dtype, static_cast<hipStream_t>(stream)));
}

lbq_status lbq_mx_matmul_workspace(const lbq_mx *a, const lbq_mx *b, size_t *bytes) {
  if (!bytes) return LBQ_ERR_NULL;
  const lbq_status st = check_matmul(a, b);
  if (st != LBQ_OK) return st;
  *bytes = scratch_bytes(dense(a->rows, b, nullptr, LBQ_F32));
  return LBQ_OK;
}

lbq_status lbq_mx_matmul(const lbq_mx *a, const lbq_mx *b, void *y, int32_t dtype, void *ws, size_t ws_bytes,
                         void *stream) {
  const lbq_status st = check_matmul(a, b);
  if (st != LBQ_OK) return st;
  if (!value_type(dtype)) return LBQ_ERR_FORMAT;
  if (a->rows == 0 || b->rows == 0) return LBQ_OK;
  MxGemm g = dense(a->rows, b, y, dtype);
  const size_t need = scratch_bytes(g);
  if (!y || (need > 0 && !ws)) return LBQ_ERR_NULL;
  if (!aligned(y, 16) || !aligned(ws, 16)) return LBQ_ERR_ALIGN;
  if (ws_bytes < need) return LBQ_ERR_WORKSPACE;
  g.a_codes = a->codes;
  g.a_scales = a->scales;
  g.scratch = ws;
  return hip_status(launch_product(g, static_cast<hipStream_t>(stream)));
}

lbq_status lbq_mx_linear_workspace(const lbq_mx *w, int32_t M, size_t *bytes) {
  if (!bytes) return LBQ_ERR_NULL;
  const lbq_status st = check_mx(w);
  if (st != LBQ_OK) return st;
  if (!mx_shape(M, w->cols)) return LBQ_ERR_SHAPE;
  *bytes = linear_layout(M, w->cols, dense(M, w, nullptr, LBQ_F16)).total;
  return LBQ_OK;
}

lbq_status lbq_mx_linear_forward(const lbq_mx *w, const void *x, int32_t M, void *y, int32_t dtype, void *ws,
                                 size_t ws_bytes, void *stream) {
  const lbq_status st = check_mx(w);
  if (st != LBQ_OK) return st;
  if (!mx_shape(M, w->cols)) return LBQ_ERR_SHAPE;
  if (!half_type(dtype)) return LBQ_ERR_FORMAT;
  if (M == 0 || w->rows == 0) return LBQ_OK;
  MxGemm g = dense(M, w, y, dtype);
  const LinearLayout l = linear_layout(M, w->cols, g);
  if (!x || !y || (l.total > 0 && !ws)) return LBQ_ERR_NULL;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(ws, 16)) return LBQ_ERR_ALIGN;
  if (ws_bytes < l.total) return LBQ_ERR_WORKSPACE;
  return quantize_and_multiply(g, x, ws, l, static_cast<hipStream_t>(stream));
}

lbq_status lbq_mx_grouped_workspace(const lbq_mx *w, int32_t E, int32_t M, int32_t T, size_t *bytes) {
  if (!bytes) return LBQ_ERR_NULL;
  const lbq_status st = check_grouped(w, E, M, T);
  if (st != LBQ_OK) return st;
  *bytes = linear_layout(M, w->cols, grouped(w, E, M, T)).total;
  return LBQ_OK;
}

lbq_status lbq_mx_grouped_forward(const lbq_mx *w, int32_t E, const void *x, int32_t M, const int32_t *offsets,
                                  const int32_t *perm, int32_t top_k, int32_t T, void *y, int32_t dtype, void *ws,
                                  size_t ws_bytes, void *stream) {
  const lbq_status st = check_grouped(w, E, M, T);
  if (st != LBQ_OK) return st;
  if (top_k < 1 || (!perm && M != T)) return LBQ_ERR_SHAPE;
  if (!half_type(dtype)) return LBQ_ERR_FORMAT;
  if (M == 0 || T == 0 || w->rows == 0) return LBQ_OK;
  if (!x || !offsets || !y) return LBQ_ERR_NULL;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(ws, 16) || !aligned(offsets, 4) || !aligned(perm, 4))
    return LBQ_ERR_ALIGN;
  MxGemm g = grouped(w, E, M, T);
  g.y = y;
  g.dtype = dtype;
  g.offsets = offsets;
  g.perm = perm;
  g.top_k = top_k;
  const LinearLayout l = linear_layout(M, w->cols, g);
  if (l.total > 0 && !ws) return LBQ_ERR_NULL;
  if (ws_bytes < l.total) return LBQ_ERR_WORKSPACE;
  return quantize_and_multiply(g, x, ws, l, static_cast<hipStream_t>(stream));
}

lbq_status lbq_moe_sort_workspace(int32_t M, int32_t E, int32_t top_k, size_t *bytes) {
  if (!bytes) return LBQ_ERR_NULL;
  const lbq_status st = check_picks(M, top_k);
  if (st != LBQ_OK) return st;
  if (E < 1 || E > kMoeMaxExperts) return LBQ_ERR_SHAPE;
  *bytes = moe_sort_ws_bytes(M * top_k, E);
  return LBQ_OK;
}

lbq_status lbq_moe_sort(const int32_t *ids, int32_t M, int32_t E, int32_t top_k, int32_t *counts, int32_t *offsets,
                        int32_t *perm, int32_t *pos, void *ws, size_t ws_bytes, void *stream) {
  const lbq_status st = check_picks(M, top_k);
  if (st != LBQ_OK) return st;
  if (E < 1 || E > kMoeMaxExperts) return LBQ_ERR_SHAPE;
  const int n = M * top_k;
  const size_t need = moe_sort_ws_bytes(n, E);
  if (!counts || !offsets || (n > 0 && (!ids || !perm || !pos)) || (need > 0 && !ws)) return LBQ_ERR_NULL;
  if (!aligned(ids, 4) || !aligned(counts, 4) || !aligned(offsets, 4) || !aligned(perm, 4) || !aligned(pos, 4) ||
      !aligned(ws, 4))
    return LBQ_ERR_ALIGN;
  if (ws_bytes < need) return LBQ_ERR_WORKSPACE;
  return hip_status(launch_moe_sort(ids, n, E, counts, offsets, perm, pos, ws, static_cast<hipStream_t>(stream)));
}

lbq_status lbq_moe_gather(const void *x, int32_t dtype, int32_t M, int32_t H, const int32_t *pos, int32_t top_k,
                          int32_t T, void *out, void *stream) {
  const lbq_status st = check_rows(dtype, M, top_k, T, H);
  if (st != LBQ_OK) return st;
  if (M == 0 || T == 0) return LBQ_OK;
  if (!x || !pos || !out) return LBQ_ERR_NULL;
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(pos, 4)) return LBQ_ERR_ALIGN;
  return hip_status(launch_moe_gather(x, dtype, M, H, T, pos, top_k, out, static_cast<hipStream_t>(stream)));
}

lbq_status lbq_moe_gather_backward(const void *d_out, int32_t dtype, int32_t T, int32_t H, const int32_t *pos,
                                   int32_t M, int32_t top_k, void *dx, void *stream) {
  const lbq_status st = check_rows(dtype, M, top_k, T, H);
  if (st != LBQ_OK) return st;
  if (M == 0) return LBQ_OK;
  if ((T > 0 && !d_out) || !pos || !dx) return LBQ_ERR_NULL;
  if (!aligned(d_out, 16) || !aligned(dx, 16) || !aligned(pos, 4)) return LBQ_ERR_ALIGN;
  return hip_status(
      launch_moe_combine(d_out, dtype, T, H, pos, nullptr, M, top_k, dx, static_cast<hipStream_t>(stream)));
}

lbq_status lbq_moe_combine(const void *o, int32_t dtype, int32_t T, int32_t H, const int32_t *pos,
                           const float *weights, int32_t M, int32_t top_k, void *y, void *stream) {
  const lbq_status st = check_rows(dtype, M, top_k, T, H);
  if (st != LBQ_OK) return st;
  if (M == 0) return LBQ_OK;
  if ((T > 0 && !o) || !pos || !weights || !y) return LBQ_ERR_NULL;
  if (!aligned(o, 16) || !aligned(y, 16) || !aligned(pos, 4) || !aligned(weights, 4)) return LBQ_ERR_ALIGN;
  return hip_status(
      launch_moe_combine(o, dtype, T, H, pos, weights, M, top_k, y, static_cast<hipStream_t>(stream)));
}

lbq_status lbq_moe_combine_backward(const void *dy, const void *o, int32_t dtype, int32_t T, int32_t H,
                                    const int32_t *pos, const float *weights, int32_t M, int32_t top_k, void *d_o,
                                    float *d_weights, void *stream) {
  const lbq_status st = check_rows(dtype, M, top_k, T, H);
  if (st != LBQ_OK) return st;
  if (M == 0) return LBQ_OK;
  if (!dy || (T > 0 && (!o || !d_o)) || !pos || !weights || !d_weights) return LBQ_ERR_NULL;
  if (!aligned(dy, 16) || !aligned(o, 16) || !aligned(d_o, 16) || !aligned(pos, 4) || !aligned(weights, 4) ||
      !aligned(d_weights, 4))
    return LBQ_ERR_ALIGN;
  return hip_status(launch_moe_combine_backward(dy, o, dtype, T, H, pos, weights, M, top_k, d_o, d_weights,
                                                static_cast<hipStream_t>(stream)));
}

}  // extern "C"
