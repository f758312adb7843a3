// Products with MX4 weights: Y = X W^T + b, W [d_o x d_i] in MX4, X in bf16 or MX4.
#include "mx4.h"

namespace qz {

namespace {

// Workgroup of four wavefronts for 16 rows of W and 16 rows of X.  The wavefronts take turns
// along d_i, 128 columns at a time: lane l has row (or token) l % 16 and the whole block
// l / 16 of the four, 16 bytes of codes with one factor.  Sums in fp32; the four partial
// sums are added in the order of the wavefronts.
constexpr int kWaves = 4;

template <bool X4>
__global__ __launch_bounds__(kWaves * 64) void mx4_product_kernel(const Mx4Product p) {
  __shared__ f32x4 part[kWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int m = lane & 15, q = lane >> 4;
  const int64_t r0 = blockIdx.x * (int64_t)16, t0 = blockIdx.y * (int64_t)16;
  const int64_t G = p.G;
  const int64_t row = r0 + m < p.d_o ? r0 + m : p.d_o - 1;
  const int64_t tok = t0 + m < p.n ? t0 + m : p.n - 1;
  const uint8_t* wc = p.codes + row * G * 16;
  const uint8_t* ws = p.scales + row * G;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int64_t st = wave; st * 4 < G; st += kWaves) {
    const int64_t b = st * 4 + q;
    const bool in = b < G;
    uint4 c = make_uint4(0u, 0u, 0u, 0u);
    uint32_t e = kMxOne;
    if (in) {
      c = *reinterpret_cast<const uint4*>(wc + b * 16);
      e = ws[b];
    }
    if constexpr (X4) {
      uint4 xc = make_uint4(0u, 0u, 0u, 0u);
      uint32_t xe = kMxOne;
      if (in) {
        xc = *reinterpret_cast<const uint4*>(p.xcodes + tok * G * 16 + b * 16);
        xe = p.xscales[tok * G + b];
      }
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
          mx_operand(c), mx_operand(xc), acc, 4, 4, 0, static_cast<int>(e), 0, static_cast<int>(xe));
    } else {
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
      const uint4* xp = reinterpret_cast<const uint4*>(p.X + tok * p.ldx + b * 32);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 xv = in ? xp[j] : make_uint4(0u, 0u, 0u, 0u);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(mx_word_bf16(w[j], mx_factor(e)),
                                                      __builtin_bit_cast(bf16x8, xv), acc, 0, 0, 0);
      }
    }
  }
  part[wave][lane] = acc;
  __syncthreads();
  if (wave != 0 || t0 + m >= p.n) return;
#pragma unroll
  for (int w = 1; w < kWaves; ++w) acc += part[w][lane];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + 4 * q + i;
    if (r >= p.d_o) break;
    const float v = p.bias ? acc[i] + p.bias[r] : acc[i];
    const int64_t at = (t0 + m) * p.ldy + r;
    if (p.yt == QZ_BF16)
      static_cast<uint16_t*>(p.Y)[at] = f32_to_bf16(v);
    else
      static_cast<float*>(p.Y)[at] = v;
  }
}

// Rows of X copied to rows of whole blocks, zero beyond d_i.
__global__ __launch_bounds__(256) void mx4_pad_kernel(const uint16_t* __restrict__ X, int64_t n,
                                                      int64_t d_i, int64_t ldx,
                                                      uint16_t* __restrict__ out, int64_t ldo) {
  for (int64_t t = blockIdx.x * (int64_t)256 + threadIdx.x; t < n * ldo;
       t += (int64_t)gridDim.x * 256) {
    const int64_t r = t / ldo, c = t % ldo;
    out[t] = c < d_i ? X[r * ldx + c] : static_cast<uint16_t>(0);
  }
}

}  // namespace

int launch_mx4_pad(const uint16_t* X, int64_t n, int64_t d_i, int64_t ldx, uint16_t* out,
                   int64_t ldo, hipStream_t s) {
  const int64_t b = ceil_div(n * ldo, 256);
  hipLaunchKernelGGL(mx4_pad_kernel, dim3(static_cast<unsigned>(b < 65536 ? b : 65536)), dim3(256),
                     0, s, X, n, d_i, ldx, out, ldo);
  return check_launch("mx4_pad");
}

int launch_mx4_product(const Mx4Product& p, hipStream_t s) {
  const dim3 g(static_cast<unsigned>(ceil_div(p.d_o, 16)), static_cast<unsigned>(ceil_div(p.n, 16)));
  if (p.X)
    hipLaunchKernelGGL((mx4_product_kernel<false>), g, dim3(kWaves * 64), 0, s, p);
  else
    hipLaunchKernelGGL((mx4_product_kernel<true>), g, dim3(kWaves * 64), 0, s, p);
  return check_launch("mx4_product");
}

}  // namespace qz
