// A routed expert layer on MX4 weights for a few tokens, in three launches:
//
//   1. logits[t][e] = <x_t, router_e>, summed in 64 bits (products of bf16 values are exact
//      there), so the choice of experts does not hang on the order of a sum.
//   2. per chosen (token t, rank r) with expert e: h = silu(g) u, [g; u] = W_gate_up[e] x_t.
//      Every workgroup finds the tokens of its expert from the logits by itself.
//   3. y_t = sum_r w_tr W_down[e_tr] h_tr, all experts of 16 output rows in one workgroup, so
//      nothing is added through memory and the order of the sums is fixed.
//
// h is kept as two bf16 numbers (value and remainder, 16 bits of mantissa together): the
// matrix cores take bf16, and rounding h once to bf16 would be as large an error as the
// final rounding of y.
#include "mx4.h"

namespace qz {

namespace {

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * 64;
constexpr int kTokens = 64;    // tokens of one workgroup of the down product

// order of the experts of a token: descending logit, ties to the lower index
__device__ __forceinline__ bool before(double a, int i, double b, int j) {
  return a > b || (a == b && i < j);
}

template <int RT>
__global__ __launch_bounds__(kThreads) void moe_logits_kernel(const MoeArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t w = blockIdx.x * (int64_t)kWaves + (threadIdx.x >> 6);
  if (w >= a.n * a.E) return;
  const int64_t t = w / a.E, e = w % a.E;
  double sum = 0;
  for (int64_t i = lane; i < a.d; i += 64)
    sum = fma(static_cast<double>(load_w<QZ_BF16>(a.X, t * a.ldx + i)),
              static_cast<double>(load_w<RT>(a.router, e * a.d + i)), sum);
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
  // a NaN sorts last, so that the choice is always k different experts
  if (lane == 0) a.logits[w] = sum == sum ? sum : -__builtin_inf();
}

__global__ __launch_bounds__(kThreads) void moe_up_kernel(const MoeArgs a) {
  __shared__ f32x4 part[2][kWaves][64];
  __shared__ int list[QZ_MOE_MAX_TOKENS];   // chosen pairs t k + r of this expert
  __shared__ int count;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int m = lane & 15, q = lane >> 4;
  const int e = blockIdx.y;
  if (threadIdx.x == 0) count = 0;
  __syncthreads();
  for (int64_t t = wave; t < a.n; t += kWaves) {
    const double* lg = a.logits + t * a.E;
    const double mine = lg[e];
    int ahead = 0;
    for (int j = lane; j < round_up(a.E, 64); j += 64)
      ahead += __popcll(__ballot(j < a.E && before(lg[j < a.E ? j : 0], j, mine, e)));
    if (ahead < a.k && lane == 0) {
      list[atomicAdd(&count, 1)] = static_cast<int>(t * a.k + ahead);
      if (blockIdx.x == 0) {
        a.sel[t * a.k + ahead] = e;
        a.top[t * a.k + ahead] = mine;
      }
    }
  }
  __syncthreads();
  const int64_t G = a.Gd, f0 = blockIdx.x * (int64_t)16;
  const int64_t row = f0 + m < a.f ? f0 + m : a.f - 1;
  const uint8_t* gc = a.gu_codes + (e * 2 * a.f + row) * G * 16;
  const uint8_t* gs = a.gu_scales + (e * 2 * a.f + row) * G;
  const uint8_t* uc = gc + a.f * G * 16;
  const uint8_t* us = gs + a.f * G;
  for (int at = 0; at < count; at += 16) {
    const int pair = list[at + m < count ? at + m : count - 1];
    const uint16_t* x = a.X + (pair / a.k) * a.ldx;
    f32x4 g = {0.f, 0.f, 0.f, 0.f}, u = g;
    for (int64_t st = wave; st * 4 < G; st += kWaves) {
      const int64_t b = st * 4 + q;
      const bool in = b < G;
      uint4 c0 = make_uint4(0u, 0u, 0u, 0u), c1 = c0;
      uint32_t e0 = kMxOne, e1 = kMxOne;
      if (in) {
        c0 = *reinterpret_cast<const uint4*>(gc + b * 16);
        c1 = *reinterpret_cast<const uint4*>(uc + b * 16);
        e0 = gs[b];
        e1 = us[b];
      }
      const uint32_t w0[4] = {c0.x, c0.y, c0.z, c0.w}, w1[4] = {c1.x, c1.y, c1.z, c1.w};
      const uint4* xp = reinterpret_cast<const uint4*>(x + b * 32);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bf16x8 xv = __builtin_bit_cast(bf16x8, in ? xp[j] : make_uint4(0u, 0u, 0u, 0u));
        g = __builtin_amdgcn_mfma_f32_16x16x32_bf16(mx_word_bf16(w0[j], mx_factor(e0)), xv, g, 0, 0, 0);
        u = __builtin_amdgcn_mfma_f32_16x16x32_bf16(mx_word_bf16(w1[j], mx_factor(e1)), xv, u, 0, 0, 0);
      }
    }
    part[0][wave][lane] = g;
    part[1][wave][lane] = u;
    __syncthreads();
    if (wave == 0 && at + m < count) {
#pragma unroll
      for (int w = 1; w < kWaves; ++w) {
        g += part[0][w][lane];
        u += part[1][w][lane];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t r = f0 + 4 * q + i;   // < 32 Gf: columns past f are zero
        const float h = r < a.f ? g[i] / (1.f + expf(-g[i])) * u[i] : 0.f;
        const uint16_t hi = f32_to_bf16(h);
        a.h_hi[pair * a.ldh + r] = hi;
        a.h_lo[pair * a.ldh + r] = f32_to_bf16(h - bf16_to_f32(hi));
      }
    }
    __syncthreads();
  }
}

__global__ __launch_bounds__(kThreads) void moe_down_kernel(const MoeArgs a) {
  __shared__ float sums[kWaves][kTokens][16];
  __shared__ float weight[kTokens * QZ_MOE_MAX_TOP_K];
  __shared__ int order[kTokens * QZ_MOE_MAX_TOP_K];
  __shared__ int start[QZ_MOE_MAX_EXPERTS + 1], fill[QZ_MOE_MAX_EXPERTS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int m = lane & 15, q = lane >> 4;
  const int64_t t0 = blockIdx.y * (int64_t)kTokens;
  const int nt = static_cast<int>(a.n - t0 < kTokens ? a.n - t0 : kTokens);
  const int pairs = nt * a.k;
  const int32_t* sel = a.sel + t0 * a.k;

  for (int i = threadIdx.x; i < a.E; i += kThreads) fill[i] = 0;
  for (int i = threadIdx.x; i < kWaves * kTokens * 16; i += kThreads) (&sums[0][0][0])[i] = 0.f;
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += kThreads) atomicAdd(&fill[sel[i]], 1);
  __syncthreads();
  if (threadIdx.x == 0) {
    int s = 0;
    for (int i = 0; i < a.E; ++i) {
      start[i] = s;
      s += fill[i];
      fill[i] = start[i];
    }
    start[a.E] = s;
  }
  __syncthreads();
  // the order of an expert's pairs is of no consequence: each is a column of its own
  for (int i = threadIdx.x; i < pairs; i += kThreads) order[atomicAdd(&fill[sel[i]], 1)] = i;
  for (int t = wave; t < nt; t += kWaves) {
    const double* top = a.top + (t0 + t) * a.k;
    const double* lg = a.logits + (t0 + t) * a.E;
    const double best = top[0];
    float s = 0.f;
    if (a.renorm) {
      for (int r = 0; r < a.k; ++r) s += expf(static_cast<float>(top[r] - best));
    } else {
      for (int j = lane; j < a.E; j += 64) s += expf(static_cast<float>(lg[j] - best));
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
    }
    if (lane < a.k) {
      const float w = expf(static_cast<float>(top[lane] - best)) / s;
      weight[t * a.k + lane] = w;
      if (blockIdx.x == 0) {
        if (a.ids) a.ids[(t0 + t) * a.k + lane] = sel[t * a.k + lane];
        if (a.weights) a.weights[(t0 + t) * a.k + lane] = w;
      }
    }
  }
  __syncthreads();

  const int64_t G = a.Gf, r0 = blockIdx.x * (int64_t)16;
  const int64_t row = r0 + m < a.d ? r0 + m : a.d - 1;
  for (int e = wave; e < a.E; e += kWaves) {
    const uint8_t* dc = a.dn_codes + (e * a.d + row) * G * 16;
    const uint8_t* ds = a.dn_scales + (e * a.d + row) * G;
    for (int at = start[e]; at < start[e + 1]; at += 16) {
      const bool mine = at + m < start[e + 1];
      const int pair = order[mine ? at + m : at];
      const uint16_t* hi = a.h_hi + (t0 * a.k + pair) * a.ldh;
      const uint16_t* lo = a.h_lo + (t0 * a.k + pair) * a.ldh;
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
      for (int64_t st = 0; st * 4 < G; ++st) {
        const int64_t b = st * 4 + q;
        const bool in = b < G;
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        uint4 c = zero;
        uint32_t f = kMxOne;
        if (in) {
          c = *reinterpret_cast<const uint4*>(dc + b * 16);
          f = ds[b];
        }
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
        const uint4* hp = reinterpret_cast<const uint4*>(hi + b * 32);
        const uint4* lp = reinterpret_cast<const uint4*>(lo + b * 32);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8 wv = mx_word_bf16(w[j], mx_factor(f));
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, __builtin_bit_cast(bf16x8, in ? hp[j] : zero), acc, 0, 0, 0);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, __builtin_bit_cast(bf16x8, in ? lp[j] : zero), acc, 0, 0, 0);
        }
      }
      if (mine)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[wave][pair / a.k][4 * q + i] += weight[pair] * acc[i];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nt * 16; i += kThreads) {
    const int t = i / 16, r = i % 16;
    if (r0 + r >= a.d) continue;
    float s = sums[0][t][r];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) s += sums[w][t][r];
    a.Y[(t0 + t) * a.d + r0 + r] = f32_to_bf16(s);
  }
}

}  // namespace

int launch_moe(const MoeArgs& a, int router_type, hipStream_t s) {
  const dim3 gl(static_cast<unsigned>(ceil_div(a.n * a.E, kWaves)));
  if (router_type == QZ_BF16)
    hipLaunchKernelGGL((moe_logits_kernel<QZ_BF16>), gl, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((moe_logits_kernel<QZ_F32>), gl, dim3(kThreads), 0, s, a);
  QZ_TRY(check_launch("moe_logits"));
  hipLaunchKernelGGL(moe_up_kernel, dim3(static_cast<unsigned>(2 * a.Gf), static_cast<unsigned>(a.E)),
                     dim3(kThreads), 0, s, a);
  QZ_TRY(check_launch("moe_up"));
  hipLaunchKernelGGL(moe_down_kernel,
                     dim3(static_cast<unsigned>(ceil_div(a.d, 16)),
                          static_cast<unsigned>(ceil_div(a.n, kTokens))),
                     dim3(kThreads), 0, s, a);
  return check_launch("moe_down");
}

}  // namespace qz
