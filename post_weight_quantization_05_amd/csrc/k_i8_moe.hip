// The routed expert layer on 8-bit integer weights: the sum over a token's experts (the products are in
// k_i8_gemm.hip and k_i8_few.hip, the sorting of pairs in i8_group.h).
#include "i8_quant.h"

namespace qz {

namespace {

// A token's results added in the order of its experts: a workgroup per 1024 columns of a token, four a
// thread; rows of y are whole fours.  Each result is added in 32 bits and rounded once.  Bound by HBM: 4096
// tokens of 6 experts, 2048 columns, 203 MB read and 17 written, 34.5 us (6.4 TB/s: some of y is still in the
// last-level cache).
__global__ __launch_bounds__(256) void i8_sum_kernel(const float* __restrict__ y, int64_t ldp,
                                                     const int32_t* __restrict__ ids, int64_t d,
                                                     int blocks, int k, int E, uint16_t* __restrict__ Y) {
  const int64_t t = blockIdx.x / static_cast<unsigned>(blocks);
  const int64_t c = (blockIdx.x % static_cast<unsigned>(blocks)) * (int64_t)1024 + 4 * threadIdx.x;
  if (c >= d) return;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int r = 0; r < k; ++r) {
    const int id = ids[t * k + r];
    if (id < 0 || id >= E) continue;
    const float4 o = *reinterpret_cast<const float4*>(y + (t * k + r) * ldp + c);
    v.x += o.x;
    v.y += o.y;
    v.z += o.z;
    v.w += o.w;
  }
  const uint2 w = make_uint2(bf16_pair(v.x, v.y), bf16_pair(v.z, v.w));
  uint16_t* const o = Y + t * d + c;
  if (d % 4 == 0 && reinterpret_cast<uintptr_t>(Y) % 8 == 0) {
    *reinterpret_cast<uint2*>(o) = w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < d) o[j] = static_cast<uint16_t>((j < 2 ? w.x : w.y) >> (16 * (j % 2)));
  }
}

}  // namespace

int launch_i8_sum(const float* y_pairs, int64_t ldp, const int32_t* ids, int64_t n, int64_t d,
                  int k, int E, uint16_t* Y, hipStream_t s) {
  const int64_t blocks = ceil_div(d, 1024);
  hipLaunchKernelGGL(i8_sum_kernel, dim3(static_cast<unsigned>(n * blocks)), dim3(256), 0, s, y_pairs, ldp, ids,
                     d, static_cast<int>(blocks), k, E, Y);
  return check_launch("i8_sum");
}

}  // namespace qz
