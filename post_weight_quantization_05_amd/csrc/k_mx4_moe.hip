// A routed expert layer on MX4 weights for a few tokens, in four launches:
//
//   1. logits[t][e] = <x_t, router_e>, summed in 64 bits (products of bf16 values are exact
//      there), so the choice of experts does not hang on the order of a sum.
//   2. per chosen (token t, rank r) with expert e: h = silu(g) u, [g; u] = W_gate_up[e] x_t.
//      Every workgroup finds its expert and that expert's tokens from the logits by itself.
//   3. the rows of W_down[e] h, per pair, fp32.
//   4. y_t = sum_r w_tr (W_down[e_tr] h_tr), in the order of r.
//
// Weights are read once per 16 tokens of an expert, 16 rows by 16 tokens on the matrix cores
// (mx4_few.h); what bounds the layer is reading them from HBM.  h is kept as two bf16 numbers
// (value and remainder, 16 bits of mantissa together): the matrix cores take bf16, and rounding h
// once to bf16 would be as large an error as the final rounding of y.  Before that rounding y is
// 2.4e-6 from 64 bits (one token, 8 of 128; relative, 2-norm) and 0.9e-7 with h in fp32; after it
// 0.00164561 either way.
//
// Measured, us (launch 2 and 3; all four): one token, 8 of 128 experts, 4096 x 1024, 54 MB: 14.3,
// 7.4; 28 to 29; 48 tokens, 6 of 64, 2048 x 1408, 294 MB: 55, 34; 96; 7 tokens, 2 of 8, 4096 x 12288,
// seven reached, 561 MB: 78, 44; 127 (92 at the 6.1 TB/s of a kernel that only reads).  Launches 1
// and 4 are 4.7 each, of which a launch alone is 3.3.
#include "mx4_few.h"

namespace qz {

namespace {

constexpr int kWaves = 8;      // of the logits' and the expert products' workgroups, at most
constexpr int kWaveLds = 4096 + 2 * 2048;   // two tiles of codes; two tiles of sums, twice
constexpr int kPerLane = QZ_MOE_MAX_EXPERTS / 64;

// order of the experts of a token: descending logit, ties to the lower index
__device__ __forceinline__ bool before(double a, int i, double b, int j) {
  return a > b || (a == b && i < j);
}

__device__ __forceinline__ void widen8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// ------------------------------------------------------------------------------ 1. the logits
// A wavefront per (token, expert), 8 columns a lane at a time.
template <int RT, bool VEC>
__global__ __launch_bounds__(256) void moe_logits_kernel(const MoeArgs a) {
  const int lane = threadIdx.x & 63;
  const int w = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (w >= a.n * a.E) return;
  const int t = w / a.E, e = w - t * a.E;
  const uint16_t* x = a.X + t * a.ldx;
  double sum = 0;
  if constexpr (VEC) {   // d % 8 = 0, both rows on 16-byte boundaries
#pragma unroll 2
    for (int64_t i = lane * 8; i < a.d; i += 512) {
      float xv[8], rv[8];
      widen8(*reinterpret_cast<const uint4*>(x + i), xv);
      if constexpr (RT == QZ_BF16) {
        widen8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.router) + e * a.d + i), rv);
      } else {
        const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(a.router) + e * a.d + i);
        const f32x4 lo = p[0], hi = p[1];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          rv[j] = lo[j];
          rv[4 + j] = hi[j];
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fma(static_cast<double>(xv[j]), static_cast<double>(rv[j]), sum);
    }
  } else {
    for (int64_t i = lane; i < a.d; i += 64)
      sum = fma(static_cast<double>(load_w<QZ_BF16>(x, i)),
                static_cast<double>(load_w<RT>(a.router, e * a.d + i)), sum);
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
  // a NaN sorts last, so that the choice is always k different experts
  if (lane == 0) a.logits[w] = sum == sum ? sum : -__builtin_inf();
}

// ------------------------------------------------------------------------- 2. gate, up, silu
// Largest of a 32-bit value over the wavefront, by data-parallel moves: lanes 1, 2, 4, 8 back in
// their rows of 16, then the last lane of a row to the next row, and of two rows to the next two.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  auto up = [](uint32_t x, uint32_t o) { return o > x ? o : x; };
  v = up(v, __builtin_amdgcn_update_dpp(0u, v, 0x111, 0xf, 0xf, false));
  v = up(v, __builtin_amdgcn_update_dpp(0u, v, 0x112, 0xf, 0xf, false));
  v = up(v, __builtin_amdgcn_update_dpp(0u, v, 0x114, 0xf, 0xf, false));
  v = up(v, __builtin_amdgcn_update_dpp(0u, v, 0x118, 0xf, 0xf, false));
  v = up(v, __builtin_amdgcn_update_dpp(0u, v, 0x142, 0xa, 0xf, false));
  v = up(v, __builtin_amdgcn_update_dpp(0u, v, 0x143, 0xc, 0xf, false));
  return __builtin_amdgcn_readlane(v, 63);
}

// The top k of one token by a wavefront, r = 0 .. k - 1 in turn: found(r, expert, logit).  Logits
// become integers of the same order and are compared upper half first.
template <class F>
__device__ __forceinline__ void wave_top_k(const double* lg, int E, int k, F found) {
  const int lane = threadIdx.x & 63;
  uint32_t hi[kPerLane], lo[kPerLane];
  bool in[kPerLane];
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    in[i] = lane + 64 * i < E;
    // -0 orders as +0
    const uint64_t b = __builtin_bit_cast(uint64_t, in[i] ? lg[lane + 64 * i] + 0.0 : 0.0);
    const uint64_t key = b >> 63 ? ~b : b | uint64_t{1} << 63;
    hi[i] = static_cast<uint32_t>(key >> 32);
    lo[i] = static_cast<uint32_t>(key);
  }
  for (int r = 0; r < k; ++r) {
    uint32_t m = 0;   // below every key
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (in[i]) m = hi[i] > m ? hi[i] : m;
    m = wave_max(m);
    uint32_t l = 0;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (in[i] && hi[i] == m) l = lo[i] > l ? lo[i] : l;
    l = wave_max(l);
    int e = -1;
#pragma unroll
    for (int i = kPerLane - 1; i >= 0; --i) {
      const uint64_t hit = __ballot(in[i] && hi[i] == m && lo[i] == l);
      if (hit) e = 64 * i + __builtin_ctzll(hit);
    }
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (lane + 64 * i == e) in[i] = false;
    const uint64_t key = static_cast<uint64_t>(m) << 32 | l;
    found(r, e, __builtin_bit_cast(double, key >> 63 ? key & ~(uint64_t{1} << 63) : ~key));
  }
}

// Workgroups (x, slot): 16 hidden columns at a time, chunks x, x + the grid's width, ...  A slot is
// an expert, or, where the tokens cannot reach all experts (`compact`), the slot-th one that they
// reach.  The first one of a slot writes its expert and pairs (t k + r) down for the launches after
// it.
__global__ __launch_bounds__(kWaves * 64, 4) void moe_up_kernel(const MoeArgs a, int compact) {
  extern __shared__ __align__(16) uint8_t smem[];   // of a wavefront: kWaveLds
  __shared__ int list[QZ_MOE_MAX_TOKENS];   // pairs of this expert
  __shared__ uint32_t reached[QZ_MOE_MAX_EXPERTS / 32];
  __shared__ int chosen[256];               // compact: n k < 256 experts
  __shared__ int count;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int m = lane & 15, q = lane >> 4;
  const bool scribe = blockIdx.x == 0;
  int e = blockIdx.y;
  if (threadIdx.x == 0) count = 0;
  if (threadIdx.x < QZ_MOE_MAX_EXPERTS / 32) reached[threadIdx.x] = 0;
  __syncthreads();
  if (compact) {
    for (int t = wave; t < a.n; t += waves)
      wave_top_k(a.logits + t * a.E, a.E, a.k, [&](int r, int c, double l) {
        if (lane != 0) return;
        chosen[t * a.k + r] = c;
        atomicOr(&reached[c / 32], 1u << (c % 32));
        if (scribe && blockIdx.y == 0) {
          a.sel[t * a.k + r] = c;
          a.top[t * a.k + r] = l;
        }
      });
    __syncthreads();
    int left = e;
    e = -1;
#pragma unroll
    for (int i = 0; i < QZ_MOE_MAX_EXPERTS / 32; ++i) {
      uint32_t bits = reached[i];
      const int here = __popc(bits);
      if (left >= 0 && left < here) {
        for (int k = 0; k < left; ++k) bits &= bits - 1;
        e = 32 * i + __builtin_ctz(bits);
      }
      left -= here;
    }
    if (e >= 0)
      for (int i = threadIdx.x; i < a.n * a.k; i += blockDim.x)
        if (chosen[i] == e) list[atomicAdd(&count, 1)] = i;
  } else {
    // eight tokens at a time: their logits are one trip to L2
    constexpr int kTogether = 8;
    for (int t0 = kTogether * wave; t0 < a.n; t0 += kTogether * waves) {
      double mine[kTogether], lg[kTogether][kPerLane];
#pragma unroll
      for (int s = 0; s < kTogether; ++s) {
        const double* row = a.logits + (t0 + s < a.n ? t0 + s : t0) * a.E;
        mine[s] = row[e];
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
          if (64 * i < a.E) lg[s][i] = row[lane + 64 * i < a.E ? lane + 64 * i : 0];
      }
#pragma unroll
      for (int s = 0; s < kTogether; ++s) {
        if (t0 + s >= a.n) break;
        int ahead = 0;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
          const int j = lane + 64 * i;
          if (64 * i < a.E) ahead += __popcll(__ballot(j < a.E && before(lg[s][i], j, mine[s], e)));
        }
        if (ahead < a.k && lane == 0) {
          const int pair = (t0 + s) * a.k + ahead;
          list[atomicAdd(&count, 1)] = pair;
          if (scribe) {
            a.sel[pair] = e;
            a.top[pair] = mine[s];
          }
        }
      }
    }
  }
  __syncthreads();
  // the order of a list is of no consequence: each pair is a column of its own
  if (scribe) {
    if (threadIdx.x == 0) {
      a.slot_expert[blockIdx.y] = e;
      a.slot_count[blockIdx.y] = count;
    }
    for (int i = threadIdx.x; i < count; i += blockDim.x) a.slot_pairs[blockIdx.y * a.n + i] = list[i];
  }
  const int G = static_cast<int>(a.Gd);
  const int n = count;
  e = __builtin_amdgcn_readfirstlane(e);
  const int units = (G + 7) / 8, mine = (units + waves - 1) / waves;
  const int u0 = wave * mine, u1 = u0 + mine < units ? u0 + mine : units;
  int turn = 0;
  auto part = [&](int w, int tile, int further = 0) -> f32x4& {
    return reinterpret_cast<f32x4*>(smem + w * kWaveLds + 4096 + turn * 2048)[tile * 64 + lane + further];
  };
  FewRows<false, 2, 1> rows;
  for (int64_t f0 = blockIdx.x * (int64_t)16; f0 < a.ldh; f0 += gridDim.x * (int64_t)16)
  for (int at = 0; at < n; at += 16) {
    const int64_t first = f0 < a.f ? f0 : a.f - 1;   // of the gate rows; the up rows follow
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      rows.codes[i] = a.gu_codes + (e * 2 * a.f + i * a.f + first) * G * 16;
      rows.scales[i] = a.gu_scales + (e * 2 * a.f + i * a.f + first) * G;
      rows.last[i] = static_cast<int>(a.f - 1 - first < 15 ? a.f - 1 - first : 15);
    }
    const bool have = at + m < n;
    const int pair = list[have ? at + m : at];
    rows.x[0][0] = reinterpret_cast<const uint8_t*>(a.X + pair / a.k * a.ldx);
    f32x4 acc[2][1] = {{f32x4{0.f, 0.f, 0.f, 0.f}}, {f32x4{0.f, 0.f, 0.f, 0.f}}};
    few_products<false, false>(rows, smem + wave * kWaveLds, G, u0, u1, acc);
    turn ^= 1;   // sums of two rounds in turn: one barrier each
    part(wave, 0) = acc[0][0];
    part(wave, 1) = acc[1][0];
    __syncthreads();
    if (wave == 0 && have) {
      f32x4 g = part(0, 0), u = part(0, 1);
      for (int w = 1; w < waves; ++w) {
        g += part(w, 0);
        u += part(w, 1);
      }
      uint16_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {   // columns past f, to the end of the last block, are zero
        const float h = f0 + 4 * q + i < a.f ? g[i] / (1.f + expf(-g[i])) * u[i] : 0.f;
        hi[i] = f32_to_bf16(h);
        lo[i] = (hi[i] & 0x7f80) == 0x7f80 ? 0 : f32_to_bf16(h - bf16_to_f32(hi[i]));   // not inf - inf
      }
      const int64_t o = pair * a.ldh + f0 + 4 * q;
      *reinterpret_cast<uint2*>(a.h_hi + o) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
      *reinterpret_cast<uint2*>(a.h_lo + o) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
    }
  }
}

// --------------------------------------------------------------------------------- 3. down
// Workgroups (x, slot), 32 rows of W_down at a time: the pairs' results, [pair][d] in fp32.  Eight
// pairs at a time: columns 0 to 7 of a tile are the values of h, 8 to 15 the remainders, and a
// result is the sum of two columns; so both halves of h cost the loads and products of one.
__global__ __launch_bounds__(kWaves * 64, 4) void moe_down_kernel(const MoeArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];   // of a wavefront: kWaveLds
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int m = lane & 15, q = lane >> 4;
  const int32_t* list = a.slot_pairs + blockIdx.y * a.n;
  // asked for together, as each is a trip to L2 (entries past the slot's count are not used)
  const int early = list[(m & 7) < a.n ? m & 7 : 0], top = list[0];
  const int n = a.slot_count[blockIdx.y];
  const int e = a.slot_expert[blockIdx.y];
  const int G = static_cast<int>(a.Gf);
  const int units = (G + 7) / 8, mine = (units + waves - 1) / waves;
  const int u0 = wave * mine, u1 = u0 + mine < units ? u0 + mine : units;
  int turn = 0;
  auto part = [&](int w, int tile, int further = 0) -> f32x4& {
    return reinterpret_cast<f32x4*>(smem + w * kWaveLds + 4096 + turn * 2048)[tile * 64 + lane + further];
  };
  FewRows<false, 2, 1> rows;
  for (int64_t r0 = blockIdx.x * (int64_t)32; r0 < a.d; r0 += gridDim.x * (int64_t)32)
  for (int at = 0; at < n; at += 8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t first = r0 + 16 * i < a.d ? r0 + 16 * i : a.d - 1;
      rows.codes[i] = a.dn_codes + (e * a.d + first) * G * 16;
      rows.scales[i] = a.dn_scales + (e * a.d + first) * G;
      rows.last[i] = static_cast<int>(a.d - 1 - first < 15 ? a.d - 1 - first : 15);
    }
    const bool have = at + (m & 7) < n;
    const int64_t pair = at == 0 ? (have ? early : top) : list[have ? at + (m & 7) : at];
    rows.x[0][0] = reinterpret_cast<const uint8_t*>((m < 8 ? a.h_hi : a.h_lo) + pair * a.ldh);
    f32x4 acc[2][1] = {{f32x4{0.f, 0.f, 0.f, 0.f}}, {f32x4{0.f, 0.f, 0.f, 0.f}}};
    few_products<false, false>(rows, smem + wave * kWaveLds, G, u0, u1, acc);
    turn ^= 1;   // sums of two rounds in turn: one barrier each
    part(wave, 0) = acc[0][0];
    part(wave, 1) = acc[1][0];
    __syncthreads();
    if (have && m < 8)
      for (int i = wave; i < 2; i += waves) {
        f32x4 v = part(0, i) + part(0, i, 8);
        for (int w = 1; w < waves; ++w) v += part(w, i) + part(w, i, 8);
        const int64_t r = r0 + 16 * i + 4 * q;
        if (r < a.ldy)   // rows of the scratch are whole fours
          *reinterpret_cast<f32x4*>(a.y_pairs + pair * a.ldy + r) = v;
      }
  }
}

// -------------------------------------------------------------------------------- 4. the sum
__global__ __launch_bounds__(256) void moe_sum_kernel(const MoeArgs a) {
  __shared__ float weight[QZ_MOE_MAX_TOP_K];
  __shared__ float sums[4];
  const int t = blockIdx.y, tid = threadIdx.x, lane = tid & 63;
  const double best = a.top[t * a.k];
  // weights: exp(l - best) over the sum of the chosen ones, or of all
  float s = 0.f;
  if (a.renorm) {
    for (int r = 0; r < a.k; ++r) s += expf(static_cast<float>(a.top[t * a.k + r] - best));
  } else {
    if (tid < a.E) s = expf(static_cast<float>(a.logits[t * a.E + tid] - best));
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
    if (lane == 0) sums[tid >> 6] = s;
    __syncthreads();
    s = sums[0] + sums[1] + sums[2] + sums[3];
  }
  if (tid < a.k) {
    const float w = expf(static_cast<float>(a.top[t * a.k + tid] - best)) / s;
    weight[tid] = w;
    if (blockIdx.x == 0) {
      if (a.ids) a.ids[t * a.k + tid] = a.sel[t * a.k + tid];
      if (a.weights) a.weights[t * a.k + tid] = w;
    }
  }
  __syncthreads();
  const int64_t c = (blockIdx.x * (int64_t)256 + tid) * 4;
  if (c >= a.d) return;
  f32x4 y = {0.f, 0.f, 0.f, 0.f};
  for (int r = 0; r < a.k; ++r)
    y += weight[r] * *reinterpret_cast<const f32x4*>(a.y_pairs + (int64_t)(t * a.k + r) * a.ldy + c);
  uint16_t* o = a.Y + t * a.d + c;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (c + i < a.d) o[i] = f32_to_bf16(y[i]);
}

}  // namespace

// Slots: one per expert, or one per pair where those are fewer and the tokens so few that every
// workgroup can find all their experts (a wavefront takes about 1 us for a token's top 8).
int moe_slots(int64_t n, int E, int k) {
  return n * k < E && n <= 2 * kWaves ? static_cast<int>(n * k) : E;
}

int launch_moe(const MoeArgs& a, int router_type, hipStream_t s) {
  const bool vec = a.d % 8 == 0 && reinterpret_cast<uintptr_t>(a.router) % 16 == 0;
  const auto logits = router_type == QZ_BF16
                          ? (vec ? moe_logits_kernel<QZ_BF16, true> : moe_logits_kernel<QZ_BF16, false>)
                          : (vec ? moe_logits_kernel<QZ_F32, true> : moe_logits_kernel<QZ_F32, false>);
  hipLaunchKernelGGL(logits, dim3(static_cast<unsigned>(ceil_div(a.n * a.E, 4))), dim3(256), 0, s, a);
  QZ_TRY(check_launch("moe_logits"));
  const unsigned slots = static_cast<unsigned>(moe_slots(a.n, a.E, a.k));
  // As many workgroups as are resident at once (four wavefronts a SIMD): finding its expert's
  // tokens takes a workgroup 1 to 2 us, so each then goes on through the rows of its slot.  As many
  // wavefronts share a chunk of rows as it takes to fill the chip, with two units or more each (one
  // where even eight do not fill it), and for finding the tokens at least two.  us, with (1, 2, 4)
  // wavefronts: 48 tokens, 6 of 64 experts, 2048 x 1408, gate and up 78, 57, 58, down 32, 35, 37; 7
  // tokens, 2 of 8, 4096 x 12288, 104, 87, 89, and 66, 49, 47.
  const auto shape = [&](int64_t chunks, int64_t G, int64_t least, dim3* grid, dim3* block) {
    const int64_t units = ceil_div(G, 8), items = chunks * slots;
    const int64_t most = items <= 512 ? units : units / 2, fill = ceil_div(256 * 16, items);
    int64_t waves = fill < kWaves ? fill : kWaves;
    if (waves > most) waves = most;
    if (waves < least) waves = least;
    if (waves < units) waves = ceil_div(units, ceil_div(units, waves));   // shares alike
    const int64_t width = ceil_div(256 * 16 / waves, slots);
    *grid = dim3(static_cast<unsigned>(chunks < width ? chunks : width), slots);
    *block = dim3(static_cast<unsigned>(64 * waves));
  };
  dim3 grid, block;
  shape(2 * a.Gf, a.Gd, 2, &grid, &block);
  hipLaunchKernelGGL(moe_up_kernel, grid, block, block.x / 64 * kWaveLds, s, a, static_cast<int>(static_cast<int>(slots) < a.E));
  QZ_TRY(check_launch("moe_up"));
  shape(ceil_div(a.d, 32), a.Gf, 1, &grid, &block);
  hipLaunchKernelGGL(moe_down_kernel, grid, block, block.x / 64 * kWaveLds, s, a);
  QZ_TRY(check_launch("moe_down"));
  hipLaunchKernelGGL(moe_sum_kernel,
                     dim3(static_cast<unsigned>(ceil_div(a.d, 1024)), static_cast<unsigned>(a.n)),
                     dim3(256), 0, s, a);
  return check_launch("moe_sum");
}

}  // namespace qz
