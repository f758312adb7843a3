// The routed expert layer on 8-bit integer weights: pairs sorted by expert, and the sum over a
// token's experts (the products are in k_i8_gemm.hip).
#include "i8_quant.h"

namespace qz {

namespace {

// Workgroup e: expert e's first slot (the pairs with smaller ids), and its pairs in their order.
// Ids outside [0, E) get no slot.
__global__ __launch_bounds__(256) void i8_group_kernel(const int32_t* __restrict__ ids, int64_t pairs,
                                                       int E, int32_t* __restrict__ offsets,
                                                       int32_t* __restrict__ order) {
  __shared__ int below[4], mine[4];
  const int e = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t part = round_up(ceil_div(pairs, 4), 64);   // a wavefront's run of pairs
  const int64_t p0 = wave * part, p1 = p0 + part < pairs ? p0 + part : pairs;
  int less = 0, same = 0;
  for (int64_t i = p0 + lane; i < p1; i += 64) {
    const int id = ids[i];
    less += id >= 0 && id < e;
    same += id == e;
  }
  for (int o = 32; o; o >>= 1) {
    less += __shfl_xor(less, o);
    same += __shfl_xor(same, o);
  }
  if (lane == 0) {
    below[wave] = less;
    mine[wave] = same;
  }
  __syncthreads();
  int at = below[0] + below[1] + below[2] + below[3];
  if (threadIdx.x == 0) {
    offsets[e] = at;
    if (e == E - 1) offsets[E] = at + mine[0] + mine[1] + mine[2] + mine[3];
  }
  for (int w = 0; w < wave; ++w) at += mine[w];
  for (int64_t i0 = p0; i0 < p1; i0 += 64) {
    const bool hit = i0 + lane < p1 && ids[i0 + lane] == e;
    const uint64_t who = __ballot(hit);
    if (hit) order[at + __popcll(who & ((uint64_t{1} << lane) - 1))] = static_cast<int32_t>(i0 + lane);
    at += __popcll(who);
  }
}

// A token's results added in the order of its experts: a workgroup per 1024 columns of a token, four a
// thread; rows of y are whole fours.
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

int launch_i8_group(const int32_t* ids, int64_t pairs, int E, int32_t* offsets, int32_t* order,
                    hipStream_t s) {
  hipLaunchKernelGGL(i8_group_kernel, dim3(E), dim3(256), 0, s, ids, pairs, E, offsets, order);
  return check_launch("i8_group");
}

int launch_i8_sum(const float* y_pairs, int64_t ldp, const int32_t* ids, int64_t n, int64_t d,
                  int k, int E, uint16_t* Y, hipStream_t s) {
  const int64_t blocks = ceil_div(d, 1024);
  hipLaunchKernelGGL(i8_sum_kernel, dim3(static_cast<unsigned>(n * blocks)), dim3(256), 0, s, y_pairs, ldp, ids,
                     d, static_cast<int>(blocks), k, E, Y);
  return check_launch("i8_sum");
}

}  // namespace qz
