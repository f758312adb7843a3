// Routing: scores, choice and weights of each token's experts, in 64 bits.
#include "qz_internal.h"

namespace qz {

namespace {

// A value and its index; the larger value wins, then the lower index.
struct Best {
  double v;
  int i;
};
__device__ __forceinline__ Best better(Best a, Best b) {
  return b.v > a.v || (b.v == a.v && b.i < a.i) ? b : a;
}
__device__ __forceinline__ Best wave_best(Best b) {
  for (int o = 32; o; o >>= 1) {
    Best c;
    c.v = __shfl_xor(b.v, o);
    c.i = __shfl_xor(b.i, o);
    b = better(b, c);
  }
  return b;
}

// A wavefront per token; lane l has the experts l, l + 64, ...
template <int LT, int PER>
__global__ __launch_bounds__(256) void route_kernel(const void* __restrict__ logits, int64_t n,
                                                    int64_t ldl, qz_router p,
                                                    const float* __restrict__ bias,
                                                    int32_t* __restrict__ ids,
                                                    float* __restrict__ weights) {
  const int lane = threadIdx.x & 63;
  const int64_t t = blockIdx.x * (int64_t)4 + (threadIdx.x >> 6);
  if (t >= n) return;
  const double none = -__builtin_inf();
  double score[PER], pick[PER];
  double top = none;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    double x = e < p.n_experts ? static_cast<double>(load_w<LT>(logits, t * ldl + e)) : none;
    if (x != x) x = none;
    score[i] = x;
    top = x > top ? x : top;
  }
  if (!(p.flags & QZ_ROUTE_SIGMOID)) {
    for (int o = 32; o; o >>= 1) top = fmax(top, __shfl_xor(top, o));
    double sum = 0.;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      pick[i] = score[i];
      score[i] = score[i] == none ? 0. : score[i] == top ? 1. : exp(score[i] - top);
      sum += score[i];
    }
    for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
    if (sum > 0.)
#pragma unroll
      for (int i = 0; i < PER; ++i) score[i] /= sum;
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      pick[i] = score[i];
      score[i] = score[i] == none ? 0. : 1. / (1. + exp(-score[i]));
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    double c = score[i];
    if (bias && e < p.n_experts) c += static_cast<double>(bias[e]);
    pick[i] = pick[i] == none || c != c ? none : c;
  }
  const int size = p.n_experts / p.n_groups;
  uint64_t kept = ~uint64_t{0};
  if (p.top_groups < p.n_groups) {
    double value = none;   // of group `lane`
    for (int g = 0; g < p.n_groups; ++g) {
      double sum = none;
      int taken = -1;
      for (int b = 0; b < p.group_best; ++b) {
        Best best{none, 1 << 20};
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int e = lane + 64 * i;
          if (e / size == g && e != taken) best = better(best, Best{pick[i], e});
        }
        best = wave_best(best);
        taken = best.i;
        if (best.v > none) sum = b == 0 ? best.v : sum + best.v;
      }
      if (lane == g) value = sum;
    }
    kept = 0;
    for (int k = 0; k < p.top_groups; ++k) {
      const bool open = lane < p.n_groups && !(kept >> lane & 1);
      const Best best = wave_best(Best{open ? value : none, open ? lane : 64 + lane});
      kept |= uint64_t{1} << (best.i & 63);
    }
  }
  // what may not be chosen sorts behind everything, by index
  int32_t my_id = 0;
  double my_w = 0.;
  uint32_t out = 0;   // bit i: expert lane + 64 i is chosen or outside
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    if (e >= p.n_experts || !(kept >> (e / size) & 1)) out |= 1u << i;
  }
  for (int k = 0; k < p.top_k; ++k) {
    Best best{none, 1 << 20};
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (!(out >> i & 1)) best = better(best, Best{pick[i], lane + 64 * i});
    best = wave_best(best);
    double w = 0.;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (best.i == lane + 64 * i) {
        out |= 1u << i;
        w = score[i];
      }
    w = __shfl(w, best.i & 63);
    if (lane == k) {
      my_id = best.i;
      my_w = w;
    }
  }
  if (p.flags & QZ_ROUTE_RENORM) {
    double sum = 0.;
    for (int k = 0; k < p.top_k; ++k) sum += __shfl(my_w, k);
    my_w = sum > 0. ? my_w / sum : 0.;
  }
  if (lane < p.top_k) {
    ids[t * p.top_k + lane] = my_id;
    weights[t * p.top_k + lane] = static_cast<float>(my_w * static_cast<double>(p.scale));
  }
}

template <int LT>
int launch_type(const void* logits, int64_t n, int64_t ldl, const qz_router& r, const float* bias,
                int32_t* ids, float* weights, hipStream_t s) {
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(ceil_div(n, 4))), dim3(256), 0, s, logits, n,
                       ldl, r, bias, ids, weights);
    return check_launch("route");
  };
  if (r.n_experts <= 64) return go(route_kernel<LT, 1>);
  if (r.n_experts <= 128) return go(route_kernel<LT, 2>);
  if (r.n_experts <= 256) return go(route_kernel<LT, 4>);
  return go(route_kernel<LT, 8>);
}

}  // namespace

int launch_route(const void* logits, int lt, int64_t n, int64_t ldl, const qz_router& r,
                 const float* bias, int32_t* ids, float* weights, hipStream_t s) {
  return lt == QZ_BF16 ? launch_type<QZ_BF16>(logits, n, ldl, r, bias, ids, weights, s)
                       : launch_type<QZ_F32>(logits, n, ldl, r, bias, ids, weights, s);
}

}  // namespace qz
