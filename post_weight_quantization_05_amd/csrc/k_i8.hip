// 8-bit integer storage: rows quantized to int8 with one scale each, and the solvers' unsigned codes
// to and from it.
#include <type_traits>

#include "qz_internal.h"

namespace qz {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// The whole number nearest to v / s (the quotient itself), ties to the even one, within +-127;
// r = 1 / s to 32 bits, so q is off by one at most.  q s - v is exact in one fused step: it is a
// multiple of both numbers' last bits' smaller one and at most s / 2 or so.
__device__ __forceinline__ float nearest_code(float v, float s, float r) {
  float q = fminf(fmaxf(__builtin_rintf(v * r), -127.f), 127.f);
  const float rest = fmaf(-q, s, v), half = 0.5f * s;
  if (fabsf(rest) > half || (fabsf(rest) == half && (static_cast<int>(q) & 1)))
    q += rest > 0.f ? 1.f : -1.f;
  return fminf(fmaxf(q, -127.f), 127.f);
}

template <int WT>
__global__ __launch_bounds__(256) void i8_quantize_kernel(
    const void* __restrict__ X, int64_t cols, int64_t ldx, const float* __restrict__ colf,
    int8_t* __restrict__ codes, float* __restrict__ scales, int32_t* __restrict__ sums,
    void* __restrict__ values) {
  __shared__ uint32_t tops[4];
  __shared__ int parts[4];
  const int64_t row = blockIdx.x, P = i8_pitch(cols);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  auto value = [&](int64_t c) {
    const float x = load_w<WT>(X, row * ldx + c);
    return colf ? x * colf[c] : x;
  };
  uint32_t top = 0;   // magnitudes compare as integers, and a NaN is above every number
  for (int64_t c = threadIdx.x; c < cols; c += 256) top = max(top, __float_as_uint(value(c)) & 0x7fffffffu);
  for (int o = 32; o; o >>= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(top, o)));
  if (lane == 0) tops[wave] = top;
  __syncthreads();
  top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
  const bool finite = top < 0x7f800000u;
  const float s = finite ? __uint_as_float(top) * (1.f / 127.f) : __uint_as_float(0x7fc00000u);
  // small rows are moved up by a power of two, exactly, so that 1 / s is a number
  const float up = s < 0x1p-60f ? 0x1p80f : 1.f, su = s * up, r = 1.f / su;
  int sum = 0;
  for (int64_t c = threadIdx.x; c < P; c += 256) {
    const float q = finite && s > 0.f && c < cols ? nearest_code(value(c) * up, su, r) : 0.f;
    codes[row * P + c] = static_cast<int8_t>(static_cast<int>(q));
    sum += static_cast<int>(q);
    if (values && c < cols) {
      if constexpr (WT == QZ_BF16)
        static_cast<uint16_t*>(values)[row * cols + c] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(q * s));
      else
        static_cast<float*>(values)[row * cols + c] = q * s;
    }
  }
  for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
  if (lane == 0) parts[wave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    scales[row] = s;
    if (sums) sums[row] = parts[0] + parts[1] + parts[2] + parts[3];
  }
}

__global__ __launch_bounds__(256) void i8_pack_kernel(const uint8_t* __restrict__ in, int64_t rows,
                                                      int64_t cols, int8_t* __restrict__ out) {
  const int64_t P = i8_pitch(cols);
  for (int64_t t = blockIdx.x * (int64_t)256 + threadIdx.x; t < rows * P; t += (int64_t)gridDim.x * 256) {
    const int64_t r = t / P, c = t % P;
    out[t] = c < cols ? static_cast<int8_t>(in[r * cols + c] ^ 0x80) : static_cast<int8_t>(0);
  }
}

__global__ __launch_bounds__(256) void i8_unpack_kernel(const int8_t* __restrict__ in, int64_t rows,
                                                        int64_t cols, uint8_t* __restrict__ out) {
  const int64_t P = i8_pitch(cols);
  for (int64_t t = blockIdx.x * (int64_t)256 + threadIdx.x; t < rows * cols; t += (int64_t)gridDim.x * 256) {
    const int64_t r = t / cols, c = t % cols;
    out[t] = static_cast<uint8_t>(in[r * P + c]) ^ 0x80;
  }
}

unsigned grid_for(int64_t items) {
  const int64_t b = ceil_div(items, 256);
  return static_cast<unsigned>(b < 65536 ? b : 65536);
}

}  // namespace

int launch_i8_quantize(const void* X, int xt, int64_t rows, int64_t cols, int64_t ldx,
                       const float* colf, int8_t* codes, float* scales, int32_t* sums, void* values,
                       hipStream_t s) {
  if (rows == 0) return QZ_OK;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(rows)), dim3(256), 0, s, X, cols, ldx, colf,
                       codes, scales, sums, values);
    return check_launch("i8_quantize");
  };
  return xt == QZ_BF16 ? go(i8_quantize_kernel<QZ_BF16>) : go(i8_quantize_kernel<QZ_F32>);
}

int launch_i8_pack(const uint8_t* codes, int64_t rows, int64_t cols, int8_t* out, hipStream_t s) {
  hipLaunchKernelGGL(i8_pack_kernel, dim3(grid_for(rows * i8_pitch(cols))), dim3(256), 0, s, codes, rows, cols, out);
  return check_launch("i8_pack");
}

int launch_i8_unpack(const int8_t* codes, int64_t rows, int64_t cols, uint8_t* out, hipStream_t s) {
  hipLaunchKernelGGL(i8_unpack_kernel, dim3(grid_for(rows * cols)), dim3(256), 0, s, codes, rows, cols, out);
  return check_launch("i8_unpack");
}

}  // namespace qz
