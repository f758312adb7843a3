// The routed expert layer on 8-bit integer weights: pairs sorted by expert, and the sum over a
// token's experts (the products are in k_i8_gemm.hip).
#include "i8_quant.h"

namespace qz {

namespace {

// Workgroup e: expert e's first slot (the pairs with smaller ids), and its pairs in their order.  Ids
// outside [0, E) get no slot.  Every workgroup reads all ids twice, four neighbours a lane, from L2: no
// counts have to pass between workgroups, and nothing depends on their order.
constexpr int kGroupWaves = 16;
__global__ __launch_bounds__(64 * kGroupWaves) void i8_group_kernel(const int32_t* __restrict__ ids,
                                                                    int64_t pairs, int E,
                                                                    int32_t* __restrict__ offsets,
                                                                    int32_t* __restrict__ order) {
  __shared__ int below[kGroupWaves], mine[kGroupWaves];
  const int e = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t part = round_up(ceil_div(pairs, kGroupWaves), 256);   // a wavefront's run of pairs
  const int64_t p0 = wave * part, p1 = p0 + part < pairs ? p0 + part : pairs;
  auto load = [&](int64_t i0, int (&id)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = i0 + 4 * lane + j;
      id[j] = i < p1 ? ids[i] : -1;
    }
  };
  int less = 0, same = 0;
#pragma unroll 2
  for (int64_t i0 = p0; i0 < p1; i0 += 256) {
    int id[4];
    load(i0, id);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      less += id[j] >= 0 && id[j] < e;
      same += id[j] == e;
    }
  }
  less = wave_sum(less);
  same = wave_sum(same);
  if (lane == 0) {
    below[wave] = less;
    mine[wave] = same;
  }
  __syncthreads();
  const int first = wave_sum(lane < kGroupWaves ? below[lane] : 0);
  if (threadIdx.x == 0) offsets[e] = first;
  if (e == E - 1 && wave == 0) {
    const int all = first + wave_sum(lane < kGroupWaves ? mine[lane] : 0);
    if (lane == 0) offsets[E] = all;
  }
  int at = first + wave_sum(lane < wave ? mine[lane] : 0);
#pragma unroll 2
  for (int64_t i0 = p0; i0 < p1; i0 += 256) {
    int id[4];
    load(i0, id);
    const uint64_t before = (uint64_t{1} << lane) - 1;
    int mark = at;   // of this lane's first hit
    int hits = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t who = __ballot(id[j] == e);
      mark += __popcll(who & before);
      hits += __popcll(who);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (id[j] == e) order[mark++] = static_cast<int32_t>(i0 + 4 * lane + j);
    at += hits;
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
  hipLaunchKernelGGL(i8_group_kernel, dim3(E), dim3(64 * kGroupWaves), 0, s, ids, pairs, E, offsets, order);
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
