// An expert layer's pairs (token, r) sorted by expert.
#pragma once

#include "i8_quant.h"

namespace qz {

// Workgroup e: expert e's first slot (the pairs with smaller ids), and its pairs in their order.  Ids
// outside [0, E) get no slot.  Every workgroup reads all ids twice, four neighbours a lane, from L2: no
// counts have to pass between workgroups, and nothing depends on their order.  4096 tokens of 6 of 64
// experts: 13.5 us together with the tokens' quantisation, whose launch it shares; with a load waited for at a
// time 17.8, with an id a lane 54.  A workgroup's own two readings are what lasts, so the time goes with the pairs and
// not with the experts: 65536 tokens of 512 columns, 8 of 64 experts 170 us, 8 of 512 161; 8192 tokens 8 of 512 22 us;
// 262144 tokens 8 of 256 595 us (quantising their hidden rows of 32 columns takes 720).
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
  // use(i0, id) for all blocks of 256 ids, four a lane; where there are kAhead of them, their loads go out together.
  constexpr int kAhead = 8;
  auto scan = [&](auto&& use) {
    int64_t i0 = p0;
    for (; vec && i0 + 256 * kAhead <= p1; i0 += 256 * kAhead) {
      int4 v[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) v[j] = *reinterpret_cast<const int4*>(ids + i0 + 256 * j + 4 * lane);
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int id[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
        use(i0 + 256 * j, id);
      }
    }
    for (; i0 < p1; i0 += 256) {
      int id[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t i = i0 + 4 * lane + j;
        id[j] = i < p1 ? ids[i] : -1;
      }
      use(i0, id);
    }
  };
  int less = 0, same = 0;
  scan([&](int64_t, const int (&id)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      less += id[j] >= 0 && id[j] < e;
      same += id[j] == e;
    }
  });
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
  const uint64_t before = (uint64_t{1} << lane) - 1;
  scan([&](int64_t i0, const int (&id)[4]) {
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
  });
}

}  // namespace qz
