// Routing: scores, choice and weights of each token's experts, in 64 bits.
#include <type_traits>

#include "qz_internal.h"

namespace qz {

namespace {

constexpr int kLanes = 16;    // of a token: exchanges stay inside a row of the vector unit
// tokens of a workgroup: their choices fit 32 KB of LDS
template <int PER>
constexpr int kRouteTokens = PER == 32 ? 8 : 16;

template <int CTRL>
__device__ __forceinline__ double row_move(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint64_t lo = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(u), CTRL, 0xf, 0xf, true));
  const uint64_t hi = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(u >> 32), CTRL, 0xf, 0xf, true));
  return __builtin_bit_cast(double, hi << 32 | lo);
}
// Largest and sum over the sixteen lanes, in each of them; a NaN counts as nothing in the former.
__device__ __forceinline__ double row_max(double v) {
  v = fmax(v, row_move<0xB1>(v));    // lane ^ 1
  v = fmax(v, row_move<0x4E>(v));    // lane ^ 2
  v = fmax(v, row_move<0x141>(v));   // mirrored in eight
  return fmax(v, row_move<0x140>(v));
}
__device__ __forceinline__ double row_sum(double v) {
  v += row_move<0xB1>(v);
  v += row_move<0x4E>(v);
  v += row_move<0x141>(v);
  return v + row_move<0x140>(v);
}

// Choices: what may be chosen but only last (a logit of -inf or NaN) sorts below every number, and
// what may not be chosen any more is a NaN, which no maximum takes and nothing equals.
constexpr double kLast = -1.7e308;
__device__ __forceinline__ double gone() { return __builtin_bit_cast(double, uint64_t{0xfff8000000000000}); }

__device__ __forceinline__ double score_of(double x, bool sigmoid, double top, double sum) {
  if (!(x > -__builtin_inf())) return 0.;
  if (sigmoid) return 1. / (1. + exp(-x));
  return sum > 0. ? (x == top ? 1. : exp(x - top)) / sum : 0.;
}

// Sixteen lanes a token, PER neighbouring experts a lane: of equal choices the lowest lane's first one
// is the lowest expert, so a choice is a maximum and a ballot.
//
// Bound by its arithmetic in 64 bits and the chain of top_k maxima.
template <int LT, int PER>
__global__ __launch_bounds__(kRouteTokens<PER> * kLanes) void route_kernel(const void* __restrict__ logits, int64_t n,
                                                    int64_t ldl, qz_router p, int vec,
                                                    const float* __restrict__ bias,
                                                    int32_t* __restrict__ ids,
                                                    float* __restrict__ weights) {
  constexpr int kTokens = kRouteTokens<PER>;
  extern __shared__ double choices[];   // [kTokens][n_experts], with groups
  __shared__ double values[kTokens][QZ_ROUTE_MAX_GROUPS];
  const int l = threadIdx.x % kLanes, in_wave = (threadIdx.x & 63) / kLanes, slot = threadIdx.x / kLanes;
  const int64_t t = blockIdx.x * (int64_t)kTokens + slot;
  const bool here = t < n;                   // every lane stays for the ballots and barriers
  const int64_t row = (here ? t : n - 1) * ldl;
  const int E = p.n_experts, e0 = l * PER;
  const double none = -__builtin_inf();
  const bool sigmoid = p.flags & QZ_ROUTE_SIGMOID;

  float x[PER];
  if (vec) {   // rows of 16 PER logits on 16-byte boundaries
    if constexpr (LT == QZ_BF16 && PER >= 8) {
#pragma unroll
      for (int i = 0; i < PER; i += 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(logits) + row + e0 + i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[i + 2 * j] = __uint_as_float(w[j] << 16);
          x[i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
      }
    } else if constexpr (LT == QZ_F32 && PER >= 4) {
#pragma unroll
      for (int i = 0; i < PER; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(logits) + row + e0 + i);
        x[i] = v.x;
        x[i + 1] = v.y;
        x[i + 2] = v.z;
        x[i + 3] = v.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) x[i] = e0 + i < E ? load_w<LT>(logits, row + e0 + i) : -__builtin_inff();
  }
  float b[PER];
  if (bias) {
#pragma unroll
    for (int i = 0; i < PER; ++i) b[i] = e0 + i < E ? bias[e0 + i] : 0.f;
  }

  double pick[PER], top = none, sum = 0.;
  if (!sigmoid) {
#pragma unroll
    for (int i = 0; i < PER; ++i) top = fmax(top, static_cast<double>(x[i]));
    top = row_max(top);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const double v = x[i];
      pick[i] = v > none ? (v == top ? 1. : exp(v - top)) : 0.;
      sum += pick[i];
    }
    sum = row_sum(sum);
    if (sum > 0.) {
#pragma unroll
      for (int i = 0; i < PER; ++i) pick[i] /= sum;
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) pick[i] = score_of(x[i], true, 0., 0.);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (bias) pick[i] += static_cast<double>(b[i]);
    if (!(x[i] > -__builtin_inff()) || !(pick[i] > none)) pick[i] = kLast;
    if (e0 + i >= E) pick[i] = gone();
  }

  if (p.top_groups < p.n_groups) {   // the same for all
    double* const mine = choices + slot * E;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (e0 + i < E) mine[e0 + i] = pick[i];
    __syncthreads();
    const int G = p.n_groups, size = E / G;
    for (int g = l; g < G; g += kLanes) {   // best and second best, the ones below every number left out
      double first = kLast, second = kLast;
      for (int i = 0; i < size; ++i) {
        const double c = mine[g * size + i];
        second = fmax(second, fmin(first, c));
        first = fmax(first, c);
      }
      values[slot][g] = p.group_best == 2 && second > kLast ? first + second : first;
    }
    __syncthreads();
    uint64_t kept = 0;   // a group stays if fewer than top_groups are better
    for (int g0 = 0; g0 < G; g0 += kLanes) {
      const int g = g0 + l;
      const double v = g < G ? values[slot][g] : none;
      int better = 0;
      for (int h = 0; h < G; ++h) {
        const double o = values[slot][h];
        better += o > v || (o == v && h < g);
      }
      const uint64_t who = __ballot(g < G && better < p.top_groups);
      kept |= (who >> (kLanes * in_wave) & 0xffff) << g0;
    }
    int g = e0 / size, left = size - e0 % size;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (!(kept >> (g & 63) & 1)) pick[i] = gone();
      if (--left == 0) {
        left = size;
        ++g;
      }
    }
  }

  double best = pick[0];
#pragma unroll
  for (int i = 1; i < PER; ++i) best = fmax(best, pick[i]);
  int my_id = 0;
  for (int k = 0; k < p.top_k; ++k) {
    const double m = row_max(best);
    const uint64_t who = __ballot(best == m) >> (kLanes * in_wave) & 0xffff;
    const int lane = __builtin_ctz(static_cast<uint32_t>(who) | 1u << kLanes);
    int id = 0;
    if (l == lane) {
      bool found = false;
      best = gone();
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const bool hit = !found && pick[i] == m;
        found = found || hit;
        id = hit ? e0 + i : id;
        pick[i] = hit ? gone() : pick[i];
        best = fmax(best, pick[i]);
      }
    }
    id = __shfl(id, lane & (kLanes - 1), kLanes);
    if (l == k) my_id = id;
  }
  // lane k has the k-th expert: its score once more
  double w = 0.;
  if (l < p.top_k) w = score_of(load_w<LT>(logits, row + my_id), sigmoid, top, sum);
  if (p.flags & QZ_ROUTE_RENORM) {
    const double total = row_sum(w);
    w = total > 0. ? w / total : 0.;
  }
  if (here && l < p.top_k) {
    ids[t * p.top_k + l] = my_id;
    weights[t * p.top_k + l] = static_cast<float>(w * static_cast<double>(p.scale));
  }
}

template <int LT>
int launch_type(const void* logits, int64_t n, int64_t ldl, const qz_router& r, const float* bias,
                int32_t* ids, float* weights, hipStream_t s) {
  const size_t size = LT == QZ_BF16 ? 2 : 4;
  auto go = [&](auto kernel, auto p) {
    constexpr int per = decltype(p)::value, tokens = kRouteTokens<per>;
    const size_t lds = r.top_groups < r.n_groups ? sizeof(double) * tokens * r.n_experts : 0;
    const int vec = r.n_experts == kLanes * per && per * size >= 16 && ldl * size % 16 == 0 &&
                    reinterpret_cast<uintptr_t>(logits) % 16 == 0;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(ceil_div(n, tokens))), dim3(tokens * kLanes), lds, s, logits, n,
                       ldl, r, vec, bias, ids, weights);
    return check_launch("route");
  };
  if (r.n_experts <= 16) return go(route_kernel<LT, 1>, std::integral_constant<int, 1>{});
  if (r.n_experts <= 32) return go(route_kernel<LT, 2>, std::integral_constant<int, 2>{});
  if (r.n_experts <= 64) return go(route_kernel<LT, 4>, std::integral_constant<int, 4>{});
  if (r.n_experts <= 128) return go(route_kernel<LT, 8>, std::integral_constant<int, 8>{});
  if (r.n_experts <= 256) return go(route_kernel<LT, 16>, std::integral_constant<int, 16>{});
  return go(route_kernel<LT, 32>, std::integral_constant<int, 32>{});
}

}  // namespace

int launch_route(const void* logits, int lt, int64_t n, int64_t ldl, const qz_router& r,
                 const float* bias, int32_t* ids, float* weights, hipStream_t s) {
  return lt == QZ_BF16 ? launch_type<QZ_BF16>(logits, n, ldl, r, bias, ids, weights, s)
                       : launch_type<QZ_F32>(logits, n, ldl, r, bias, ids, weights, s);
}

}  // namespace qz
