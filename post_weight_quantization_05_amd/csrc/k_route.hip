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

// a b + c with c in scalar registers: the compiler's accumulating form would first copy c.
__device__ __forceinline__ double fma_const(double a, double b, double c) {
  double d;
  asm("v_fma_f64 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "s"(c));
  return d;
}

// e^v: v = n ln 2 + r with |r| <= ln 2 / 2, and the power series of e^r up to r^13 / 13! (the next term
// is below 2^-57).  Off by a last bit or two; 0 and infinity where 64 bits end.
__device__ __forceinline__ double exp64(double v) {
  v = fmin(fmax(v, -1000.), 1000.);
  const double n = __builtin_rint(v * 1.4426950408889634074);
  // ln 2 in two parts, the first of 32 bits, so that n times it is exact
  double r = fma(-n, 0x1.62e42feep-1, v);
  r = fma(-n, 0x1.a39ef35793c76p-33, r);
  double e = fma_const(r, 1. / 6227020800., 1. / 479001600.);
  e = fma_const(e, r, 1. / 39916800.);
  e = fma_const(e, r, 1. / 3628800.);
  e = fma_const(e, r, 1. / 362880.);
  e = fma_const(e, r, 1. / 40320.);
  e = fma_const(e, r, 1. / 5040.);
  e = fma_const(e, r, 1. / 720.);
  e = fma_const(e, r, 1. / 120.);
  e = fma_const(e, r, 1. / 24.);
  e = fma_const(e, r, 1. / 6.);
  e = fma(e, r, 0.5);
  e = fma(e, r, 1.);
  e = fma(e, r, 1.);
  return __builtin_ldexp(e, static_cast<int>(n));
}

// Scores: 0 for a logit of -inf or NaN.
__device__ __forceinline__ double sigmoid64(double x) {
  const double s = 1. / (1. + exp64(-x));
  return x > -__builtin_inf() ? s : 0.;
}
__device__ __forceinline__ double softmax64(double x, double top) {   // before it is divided by the sum
  const double e = exp64(x - top);
  return x > -__builtin_inf() ? (x == top ? 1. : e) : 0.;
}

// Sixteen lanes a token, PER neighbouring experts a lane: of equal choices the lowest lane's first one
// is the lowest expert, so a choice is a maximum and a ballot.
//
// Scores and choices are held in 64 bits, so that two experts change places only where their choices
// differ by less than a score's last bits.  Bound by that arithmetic (an exponential and a quotient an
// expert) and by the chain of top_k maxima with a lane's choices looked through after each, of which two wavefronts a
// SIMD (8192 tokens) cover little: 8192 tokens, 256 experts in 8 groups, fp32, 14 us, where the logits' 8.4 MB alone
// would take 1.7; one token of 128, 5.1 us: the launch, and one wavefront's chain of that arithmetic.
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
      pick[i] = softmax64(x[i], top);
      sum += pick[i];
    }
    sum = row_sum(sum);
    if (sum > 0.) {
#pragma unroll
      for (int i = 0; i < PER; ++i) pick[i] /= sum;
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) pick[i] = sigmoid64(x[i]);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (bias) pick[i] += static_cast<double>(b[i]);
    if (!(x[i] > -__builtin_inff()) || !(pick[i] > none)) pick[i] = kLast;
    if (e0 + i >= E) pick[i] = gone();
  }

  const int G = p.n_groups, size = E / G, span = size / PER;   // lanes of a group, where they are whole
  if (p.top_groups < G && size % PER == 0 && (span & (span - 1)) == 0) {   // the same for all
    // A lane's experts are of one group, and so are `span` neighbouring lanes: all in registers.  (Lanes
    // past the experts have no group and are not asked.)
    double first = kLast, second = kLast;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      second = fmax(second, fmin(first, pick[i]));
      first = fmax(first, pick[i]);
    }
    for (int o = 1; o < span; o *= 2) {
      const double f = __shfl_xor(first, o), c = __shfl_xor(second, o);
      second = fmax(fmax(second, c), fmin(first, f));
      first = fmax(first, f);
    }
    const double v = p.group_best == 2 && second > kLast ? first + second : first;
    const int g = l / span;
    int better = 0;
    for (int h = 0; h < G; ++h) {
      const double o = __shfl(v, h * span, kLanes);
      better += o > v || (o == v && h < g);
    }
    if (better >= p.top_groups)
#pragma unroll
      for (int i = 0; i < PER; ++i) pick[i] = gone();
  } else if (p.top_groups < G) {
    double* const mine = choices + slot * E;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (e0 + i < E) mine[e0 + i] = pick[i];
    __syncthreads();
    for (int g = l; g < G; g += kLanes) {   // best and second best, the ones below every number left out
      double first = kLast, second = kLast;
#pragma unroll 4
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

  auto largest = [&] {   // in four chains
    double m[4] = {pick[0], gone(), gone(), gone()};
#pragma unroll
    for (int i = 1; i < PER; ++i) m[i % 4] = fmax(m[i % 4], pick[i]);
    return PER > 2 ? fmax(fmax(m[0], m[1]), fmax(m[2], m[3])) : fmax(m[0], m[1]);
  };
  double best = largest();
  int my_id = 0;
  for (int k = 0; k < p.top_k; ++k) {
    const double m = row_max(best);
    const uint64_t who = __ballot(best == m) >> (kLanes * in_wave) & 0xffff;
    const int lane = __builtin_ctz(static_cast<uint32_t>(who) | 1u << kLanes);
    int id = 0;
    if (l == lane) {
#pragma unroll
      for (int i = PER - 1; i >= 0; --i) id = pick[i] == m ? i : id;
#pragma unroll
      for (int i = 0; i < PER; ++i) {   // the high word makes it a NaN
        const uint64_t u = __builtin_bit_cast(uint64_t, pick[i]);
        const uint32_t hi = i == id ? 0xfff80000u : static_cast<uint32_t>(u >> 32);
        pick[i] = __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | static_cast<uint32_t>(u));
      }
      best = largest();
      id += e0;
    }
    id = __shfl(id, lane & (kLanes - 1), kLanes);
    if (l == k) my_id = id;
  }
  // lane k has the k-th expert: its score once more
  double w = 0.;
  if (l < p.top_k) {
    const double v = load_w<LT>(logits, row + my_id);
    w = sigmoid ? sigmoid64(v) : sum > 0. ? softmax64(v, top) / sum : 0.;
  }
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
