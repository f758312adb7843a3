// Microscaled 4-bit (MX4) quantisation: round-to-nearest of a matrix on E2M1 elements with
// one power-of-two factor per 32 columns of a row.
#include "mx4.h"

namespace qz {

namespace {

constexpr int kThreads = 256;

template <int WT>
__global__ __launch_bounds__(kThreads) void mx4_quantize_kernel(
    const void* __restrict__ W, int64_t rows, int64_t cols, int64_t ldw, int least,
    const float* __restrict__ colw, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
    void* __restrict__ values) {
  const int64_t G = mx_blocks(cols);
  for (int64_t t = blockIdx.x * (int64_t)kThreads + threadIdx.x; t < rows * G;
       t += (int64_t)gridDim.x * kThreads) {
    const int64_t r = t / G, c0 = (t % G) * kMxBlock;
    float v[kMxBlock];
    uint32_t top = 0;   // magnitudes compare as integers; a NaN is above every number
#pragma unroll
    for (int i = 0; i < kMxBlock; ++i) {
      v[i] = c0 + i < cols ? load_w<WT>(W, r * ldw + c0 + i) : 0.f;
      const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
      top = b > top ? b : top;
    }
    const uint32_t ex = top >> 23;
    const bool bad = ex == 255;
    uint32_t e = ex > 2 ? ex - 2 : 0;
    if (bad) e = 255;
    if (least && !bad) {
      double d0 = 0, d1 = 0;
#pragma unroll
      for (int i = 0; i < kMxBlock; i += 2) {
        const uint32_t q0 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[i], v[i + 1], mx_factor(e), 0);
        const uint32_t q1 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[i], v[i + 1], mx_factor(e + 1), 0);
        const auto x0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q0, mx_factor(e), 0);
        const auto x1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q1, mx_factor(e + 1), 0);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const double h = c0 + i + j < cols ? (colw ? (double)colw[c0 + i + j] : 1.0) : 0.0;
          const double a = (double)v[i + j] - (double)x0[j], b = (double)v[i + j] - (double)x1[j];
          d0 += a * a * h;
          d1 += b * b * h;
        }
      }
      if (d1 < d0) e += 1;
    }
    uint32_t word[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kMxBlock; i += 2) {
      uint32_t q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[i], v[i + 1], mx_factor(e), 0);
      if (bad) q = 0;
      word[i / 8] |= q << (4 * (i % 8));
      if (values) {
        const auto x = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, mx_factor(e), 0);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (c0 + i + j < cols) {
            if constexpr (WT == QZ_BF16)
              static_cast<uint16_t*>(values)[r * cols + c0 + i + j] = f32_to_bf16(x[j]);
            else
              static_cast<float*>(values)[r * cols + c0 + i + j] = x[j];
          }
      }
    }
    *reinterpret_cast<uint4*>(codes + t * 16) = make_uint4(word[0], word[1], word[2], word[3]);
    scales[t] = static_cast<uint8_t>(e);
  }
}

// One thread per block: the codes as integers 2 x (E2M1 value) and the factor halved, which
// is qz_objective_i32's form of the same numbers (zero point 0).
__global__ __launch_bounds__(kThreads) void mx4_unpack_kernel(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows,
    int64_t cols, int32_t* __restrict__ out, float* __restrict__ out_scales,
    uint8_t* __restrict__ zeros) {
  const int64_t G = mx_blocks(cols);
  for (int64_t t = blockIdx.x * (int64_t)kThreads + threadIdx.x; t < rows * G;
       t += (int64_t)gridDim.x * kThreads) {
    const int64_t r = t / G, c0 = (t % G) * kMxBlock;
    const uint4 c = *reinterpret_cast<const uint4*>(codes + t * 16);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < kMxBlock; ++i) {
      const uint32_t q = (w[i / 8] >> (4 * (i % 8))) & 15u;
      // magnitude codes 0..7 -> 0 1 2 3 4 6 8 12, four bits each
      const int mag = static_cast<int>((0xC8643210u >> (4 * (q & 7u))) & 15u);
      if (c0 + i < cols) out[r * cols + c0 + i] = (q & 8u) ? -mag : mag;
    }
    const uint32_t e = scales[t];
    // 2^(e - 128): below e = 2 a subnormal number
    out_scales[t] = e == 255 ? __uint_as_float(0x7fc00000u)
                             : __uint_as_float(e >= 2 ? (e - 1) << 23 : 1u << (21 + e));
    zeros[t] = 0;
  }
}

int grid_for(int64_t items) {
  const int64_t b = ceil_div(items, kThreads);
  return static_cast<int>(b < (1 << 20) ? b : (1 << 20));
}

}  // namespace

int launch_mx4_quantize(const void* W, int wt, int64_t rows, int64_t cols, int64_t ldw, int rule,
                        const float* colw, uint8_t* codes, uint8_t* scales, void* values,
                        hipStream_t s) {
  const int least = rule == QZ_MX4_LEAST;
  const dim3 g(grid_for(rows * mx_blocks(cols)));
  if (wt == QZ_BF16)
    hipLaunchKernelGGL((mx4_quantize_kernel<QZ_BF16>), g, dim3(kThreads), 0, s, W, rows, cols, ldw,
                       least, colw, codes, scales, values);
  else
    hipLaunchKernelGGL((mx4_quantize_kernel<QZ_F32>), g, dim3(kThreads), 0, s, W, rows, cols, ldw,
                       least, colw, codes, scales, values);
  return check_launch("mx4_quantize");
}

int launch_mx4_unpack(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                      int32_t* out, float* out_scales, uint8_t* zeros, hipStream_t s) {
  hipLaunchKernelGGL(mx4_unpack_kernel, dim3(grid_for(rows * mx_blocks(cols))), dim3(kThreads), 0,
                     s, codes, scales, rows, cols, out, out_scales, zeros);
  return check_launch("mx4_unpack");
}

}  // namespace qz
