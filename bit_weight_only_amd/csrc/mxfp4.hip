// MXFP4 tensors: quantisation along rows or columns, and the values back.
//
// A block is 32 values along the axis a product will sum over. With m the
// block's largest magnitude, e = clamp(floor(log2 m) - 2, -127, 125) (-127 for
// m = 0) and a value is held as e2m1(x / 2^e): round to nearest, ties to the
// even code, magnitudes past 6 saturated (the largest is below 8). The scale
// byte is e + 127 (E8M0). A block with a NaN or an infinity has byte 255 and
// zero codes; everything it meets in a product is NaN.
//
// Exact throughout: the division is by a power of two inside the conversion
// instruction (v_cvt_scalef32_pk_fp4_*: rounds once, saturates, keeps signs,
// takes the subnormal scale 2^-127), so codes are bit-equal to the definition.
//
// Bound: HBM. 16-bit input moves 2 + 17/32 bytes per value and a lane spends
// about two instructions per value. 16384 x 4096 bf16: quantized in 30 us, 5.6
// TB/s; the values back in 27 us, 6.2 TB/s.
#include "device.h"
#include "kernels.h"
#include "mxfp4.h"

namespace lbq {

namespace {

using namespace mxfp4;

constexpr int kThreads = 256;

// Eight consecutive values of a row as they come from memory.
template <int DT>
struct In {
  uint4 v;
  static __device__ __forceinline__ In load(const void *p, size_t unit) {
    return In{static_cast<const uint4 *>(p)[unit]};
  }
  __device__ __forceinline__ uint32_t mag() const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
    return m;
  }
  __device__ __forceinline__ uint32_t codes(float s) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    return codes8<DT>(w, s);
  }
};
template <>
struct In<kF32> {
  float4_t a, b;
  static __device__ __forceinline__ In load(const void *p, size_t unit) {
    return In{static_cast<const float4_t *>(p)[2 * unit], static_cast<const float4_t *>(p)[2 * unit + 1]};
  }
  __device__ __forceinline__ uint32_t mag() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m = max(m, max(__float_as_uint(a[i]) & 0x7FFFFFFFu, __float_as_uint(b[i]) & 0x7FFFFFFFu));
    return m;
  }
  __device__ __forceinline__ uint32_t codes(float s) const {
    const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    return codes8_f32(v, s);
  }
};

// ------------------------------------------------------------------ along rows

// Four lanes per block, eight values each: sixteen lanes make one 128-group of
// one row, whose four scale bytes leave as one word. Unit u is eight values;
// group u / 16.
template <int DT>
__global__ void __launch_bounds__(kThreads) mx_quantize_kernel(const void *__restrict__ x, uint32_t *__restrict__ codes,
                                                               uint32_t *__restrict__ scales, int rows,
                                                               uint32_t groups, long units) {
  const long step = static_cast<long>(gridDim.x) * kThreads;
  // units is a multiple of 16, so the sixteen lanes of a group stay together
  for (long u = static_cast<long>(blockIdx.x) * kThreads + threadIdx.x; u < units; u += step) {
    const In<DT> in = In<DT>::load(x, static_cast<size_t>(u));
    uint32_t m = in.mag();
    m = max(m, xor_lane_u32<1>(m));
    m = max(m, xor_lane_u32<2>(m));
    const uint32_t byte = scale_byte<DT>(m);
    const uint32_t c = in.codes(scale_value(byte));
    codes[u] = byte == 255u ? 0u : c;
    uint32_t word = byte << (8 * ((threadIdx.x >> 2) & 3));
    word |= xor_lane_u32<4>(word);
    word |= xor_lane_u32<8>(word);
    if ((threadIdx.x & 15) == 0) {
      const uint32_t gi = static_cast<uint32_t>(u >> 4), row = gi / groups;   // fewer than 2^31 groups
      scales[static_cast<size_t>(gi - row * groups) * rows + row] = word;
    }
  }
}

// ------------------------------------------------------------------ along columns

// The transposed tensor: blocks of 32 rows of x. A workgroup takes 128 rows by
// 256 bytes of columns (128 columns in 16 bits, 64 in fp32) through LDS, rows of
// 64 words. Wave b then owns rows 32 b .. 32 b + 31 and lane l the column, or
// pair of columns, of word l: a read of one row by the wave is 64 neighbouring
// words. Codes leave through LDS too, so that the four 16-byte blocks of a
// column go out side by side. Rows and columns past the end count as zeros.
//
// Bound: HBM (2 + 17/32 bytes per 16-bit value). 8192 x 14336 bf16 73 us, 4.1
// TB/s. VEC: every row starts on a 16-byte boundary.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) mx_quantize_t_kernel(const void *__restrict__ x, uint4 *__restrict__ codes,
                                                                 uint32_t *__restrict__ scales, int rows, int cols,
                                                                 int row_groups) {
  using T = typename Elem<DT>::type;
  constexpr int kPer = DT == kF32 ? 1 : 2;        // columns per word
  constexpr int kCols = 64 * kPer, kVec = 4 * kPer;   // of a tile; of 16 bytes
  __shared__ __attribute__((aligned(16))) uint32_t tile[128][64];
  __shared__ __attribute__((aligned(4))) uint8_t bytes[kCols][4];
  const int c0 = blockIdx.x * kCols, g = blockIdx.y;
  const T *src = static_cast<const T *>(x);
#pragma unroll
  for (int it = 0; it < 8; ++it) {
    const int i = it * kThreads + threadIdx.x, r = i >> 4, c = c0 + (i & 15) * kVec;
    const int row = min(g * 128 + r, rows - 1);
    const bool there = g * 128 + r < rows;
    uint4 v = make_uint4(0, 0, 0, 0);
    if constexpr (VEC) {
      if (there && c < cols) v = *reinterpret_cast<const uint4 *>(src + static_cast<size_t>(row) * cols + c);
    } else {
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < kVec; ++e)
        if (there && c + e < cols) {
          const T t = src[static_cast<size_t>(row) * cols + c + e];
          if constexpr (DT == kF32) w[e] = __float_as_uint(t);
          else w[e / 2] |= static_cast<uint32_t>(t) << (16 * (e % 2));
        }
      v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    *reinterpret_cast<uint4 *>(&tile[r][4 * (i & 15)]) = v;
  }
  __syncthreads();
  const int l = threadIdx.x & 63, b = threadIdx.x >> 6;
  uint32_t w[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) w[i] = tile[32 * b + i][l];
  __syncthreads();   // the tile's words are read: its memory takes the codes
  uint4 *out = reinterpret_cast<uint4 *>(&tile[0][0]);   // [kCols][4]
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    uint32_t m = 0, byte;
    uint32_t o[4];
    if constexpr (DT == kF32) {
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        v[i] = __uint_as_float(w[i]);
        m = max(m, w[i] & 0x7FFFFFFFu);
      }
      byte = scale_byte<DT>(m);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = codes8_f32(v + 8 * i, scale_value(byte));
    } else {
      // this column's 16-bit values, two rows to a word
      uint32_t v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        v[i] = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], p == 0 ? 0x05040100u : 0x07060302u);
        m = max(m, max(v[i] & 0x7FFFu, (v[i] >> 16) & 0x7FFFu));
      }
      byte = scale_byte<DT>(m);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = codes8<DT>(v + 4 * i, scale_value(byte));
    }
    const int c = kPer * l + p;
    out[c * 4 + b] = byte == 255u ? make_uint4(0, 0, 0, 0) : make_uint4(o[0], o[1], o[2], o[3]);
    bytes[c][b] = static_cast<uint8_t>(byte);
  }
  __syncthreads();
#pragma unroll
  for (int it = 0; it < kCols * 4 / kThreads; ++it) {
    const int i = it * kThreads + threadIdx.x, c = c0 + (i >> 2);
    if (c < cols) codes[(static_cast<size_t>(c) * row_groups + g) * 4 + (i & 3)] = out[i];
  }
  const int c = threadIdx.x;
  if (c < kCols && c0 + c < cols)
    scales[static_cast<size_t>(g) * cols + c0 + c] = *reinterpret_cast<const uint32_t *>(bytes[c]);
}

// ------------------------------------------------------------------ values

template <int DT>
__global__ void __launch_bounds__(kThreads) mx_dequantize_kernel(const uint32_t *__restrict__ codes,
                                                                 const uint32_t *__restrict__ scales,
                                                                 void *__restrict__ out, int rows, uint32_t groups,
                                                                 long units) {
  const long step = static_cast<long>(gridDim.x) * kThreads;
  for (long u = static_cast<long>(blockIdx.x) * kThreads + threadIdx.x; u < units; u += step) {
    const uint32_t gi = static_cast<uint32_t>(u >> 4), row = gi / groups;
    const uint32_t word = scales[static_cast<size_t>(gi - row * groups) * rows + row];
    const uint32_t byte = (word >> (8 * ((u >> 2) & 3))) & 0xFFu;
    const float s = byte == 255u ? __uint_as_float(0x7FC00000u) : scale_value(byte);
    const uint32_t c = codes[u];
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = s * e2m1_value((c >> (4 * i)) & 15u);
    store8<DT>(out, static_cast<size_t>(u), v);
  }
}

int grid_of(long units) {
  const long g = (units + kThreads - 1) / kThreads;
  return static_cast<int>(g < 16384 ? g : 16384);
}

}  // namespace

hipError_t launch_mx_quantize(const void *x, int dtype, int rows, int cols, void *codes, void *scales, hipStream_t s) {
  const long units = static_cast<long>(rows) * cols / 8;
  const int grid = grid_of(units), groups = cols / kGroup;
  uint32_t *c = static_cast<uint32_t *>(codes), *e = static_cast<uint32_t *>(scales);
  if (dtype == kF16)
    hipLaunchKernelGGL(mx_quantize_kernel<kF16>, dim3(grid), dim3(kThreads), 0, s, x, c, e, rows, groups, units);
  else if (dtype == kBF16)
    hipLaunchKernelGGL(mx_quantize_kernel<kBF16>, dim3(grid), dim3(kThreads), 0, s, x, c, e, rows, groups, units);
  else
    hipLaunchKernelGGL(mx_quantize_kernel<kF32>, dim3(grid), dim3(kThreads), 0, s, x, c, e, rows, groups, units);
  return hipGetLastError();
}

hipError_t launch_mx_quantize_t(const void *x, int dtype, int rows, int cols, void *codes, void *scales,
                                hipStream_t s) {
  const int rg = static_cast<int>((static_cast<long>(rows) + 127) / 128);
  const int per = dtype == kF32 ? 64 : 128;
  const dim3 grid((cols + per - 1) / per, rg);
  const bool vec = cols % (dtype == kF32 ? 4 : 8) == 0;
  uint4 *c = static_cast<uint4 *>(codes);
  uint32_t *e = static_cast<uint32_t *>(scales);
#define LBQ_MX_GO(DT)                                                                                               \
  if (vec) hipLaunchKernelGGL((mx_quantize_t_kernel<DT, true>), grid, dim3(kThreads), 0, s, x, c, e, rows, cols, rg); \
  else hipLaunchKernelGGL((mx_quantize_t_kernel<DT, false>), grid, dim3(kThreads), 0, s, x, c, e, rows, cols, rg)
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

hipError_t launch_mx_dequantize(const void *codes, const void *scales, int rows, int cols, void *out, int dtype,
                                hipStream_t s) {
  const long units = static_cast<long>(rows) * cols / 8;
  const int grid = grid_of(units), groups = cols / kGroup;
  const uint32_t *c = static_cast<const uint32_t *>(codes), *e = static_cast<const uint32_t *>(scales);
  if (dtype == kF16)
    hipLaunchKernelGGL(mx_dequantize_kernel<kF16>, dim3(grid), dim3(kThreads), 0, s, c, e, out, rows, groups, units);
  else if (dtype == kBF16)
    hipLaunchKernelGGL(mx_dequantize_kernel<kBF16>, dim3(grid), dim3(kThreads), 0, s, c, e, out, rows, groups, units);
  else
    hipLaunchKernelGGL(mx_dequantize_kernel<kF32>, dim3(grid), dim3(kThreads), 0, s, c, e, out, rows, groups, units);
  return hipGetLastError();
}

}  // namespace lbq
