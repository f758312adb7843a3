// An expert layer's pairs (token, r) sorted by expert.
#pragma once

#include "i8_quant.h"

namespace qz {

// Workgroup e: expert e's first slot (the pairs with smaller ids), and its pairs in their order.  Ids
// outside [0, E) get no slot.  Every workgroup reads all ids twice, four neighbours a lane, from L2: no
// counts have to pass between workgroups, and nothing depends on their order.  4096 tokens of 6 of 64
// experts: 18.6 us together with the tokens' quantisation, whose launch it shares; with an id a lane 54 us.
struct Grouping {
  const int32_t* ids;
  int64_t pairs;
  int E;
  int32_t* offsets;   // [E + 1]
  int32_t* order;     // [pairs]
};
template <int WAVES>
__device__ __forceinline__ void group_expert(const Grouping& g, int e) {
  __shared__ int below[WAVES], mine[WAVES];
  const int32_t* const ids = g.ids;
  const int64_t pairs = g.pairs;
  const int E = g.E;
  int32_t* const offsets = g.offsets;
  int32_t* const order = g.order;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t part = round_up(ceil_div(pairs, WAVES), 256);   // a wavefront's run of pairs
  const int64_t p0 = wave * part, p1 = p0 + part < pairs ? p0 + part : pairs;
  const bool vec = reinterpret_cast<uintptr_t>(ids) % 16 == 0;
  auto load = [&](int64_t i0, int (&id)[4]) {
    if (vec && i0 + 256 <= p1) {
      const int4 v = *reinterpret_cast<const int4*>(ids + i0 + 4 * lane);
      id[0] = v.x;
      id[1] = v.y;
      id[2] = v.z;
      id[3] = v.w;
      return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = i0 + 4 * lane + j;
      id[j] = i < p1 ? ids[i] : -1;
    }
  };
  int less = 0, same = 0;
#pragma unroll 4
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
  const int first = wave_sum(lane < WAVES ? below[lane] : 0);
  if (threadIdx.x == 0) offsets[e] = first;
  if (e == E - 1 && wave == 0) {
    const int all = first + wave_sum(lane < WAVES ? mine[lane] : 0);
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

}  // namespace qz
