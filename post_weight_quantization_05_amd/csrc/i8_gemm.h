// Products of 8-bit integer rows, shared by the tile kernels and the few-token kernels: where a
// workgroup's rows lie, and how an integer sum becomes a result.
#pragma once

#include <atomic>

#include "i8_quant.h"

namespace qz {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

enum Form { kPlain, kGateUp, kDown };

enum class I8Kind;
int launch_i8_few(I8Kind kind, int form, const I8Product& p, hipStream_t s);

// An integer sum with its zero point, scales and bias.  shift: the zero point less 128; -2^23 <= xsum < 2^23
// (65536 codes), so the product takes the 24-bit multiplier.
__device__ __forceinline__ float scaled(int a, int shift, int xsum, float sx, float sw, float bias) {
  return fmaf(static_cast<float>(a - __mul24(shift, xsum)) * sx, sw, bias);
}

// silu: g / (1 + e^-g), off by less than 8 2^-24 of itself, and half of 2^-149 where it is below 2^-126.
//
// Up to |g| = 80, where neither the power nor its sum with 1 leaves the normal numbers: e^-g = 2^h e^(-g - h ln 2)
// with h = -g log2 e rounded.  The hardware's power of two and reciprocal are a last bit off (2 2^-24 each), the second
// factor is 1 + its exponent, below 2^-17, with ln 2 in two parts; its step, the sum and the product round once each.
__device__ __forceinline__ float silu_near(float g) {
  const float h = -0x1.715476p+0f * g, e = __builtin_amdgcn_exp2f(h);
  const float rest = fmaf(h, 0x1.05c61p-29f, fmaf(h, -0x1.62e43p-1f, -g));
  return g * __builtin_amdgcn_rcpf(1.f + fmaf(e, rest, e));
}
// Beyond: g itself, or g e^g = g p 2^n with n whole and p the power of two of a fraction within +-1/2, 2^n put on
// at the end.  (Below -256 it is zero.)
__device__ __forceinline__ float silu_far(float g) {
  const float a = fminf(fabsf(g), 256.f), n = __builtin_rintf(-0x1.715476p+0f * a);
  const float p = __builtin_amdgcn_exp2f(fmaf(-0x1.4ae0cp-26f, a, fmaf(-0x1.715476p+0f, a, -n)));
  return g < 0.f ? __builtin_ldexpf(g * p, static_cast<int>(n)) : g;
}
__device__ __forceinline__ float silu(float g) {
  const float v = silu_near(g);
  return fabsf(g) > 80.f ? silu_far(g) : v;
}
// Of four, with one look at whether any of the wavefront's is far.  (A large tile ends with 64 of them a thread: 4096
// tokens 6 of 64, 2048 -> 2 x 1408, gate and up 209 us in a warm loop, 207 by the plain form, which overflows and loses
// |g| last bits; 221 with a power split for every g.)
__device__ __forceinline__ f32x4 silu(const f32x4& g) {
  f32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = silu_near(g[i]);
  const float most = fmaxf(fmaxf(fabsf(g[0]), fabsf(g[1])), fmaxf(fabsf(g[2]), fabsf(g[3])));
  if (__ballot(most > 80.f)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fabsf(g[i]) > 80.f ? silu_far(g[i]) : v[i];
  }
  return v;
}

// The token tiles of `bn` slots of an expert layer, the experts' tiles in their order.  Every lane of a
// wavefront has eight neighbouring experts.
struct Tiles {
  int at[9], upto, tiles;   // the lane's experts' slots; tiles up to and of the lane
  int total;
  __device__ __forceinline__ Tiles(const I8Product& p, int bn) {
    const int lane = threadIdx.x & 63;
    tiles = 0;
#pragma unroll
    for (int i = 0; i <= 8; ++i) {
      const int e = 8 * lane + i;
      at[i] = p.offsets[e < p.E ? e : p.E];
      if (i) tiles += (at[i] - at[i - 1] + bn - 1) / bn;
    }
    upto = tiles;
    for (int o = 1; o < 64; o *= 2) {
      const int v = __shfl_up(upto, o);
      if (lane >= o) upto += v;
    }
    total = __builtin_amdgcn_readlane(upto, 63);
  }
  // Expert and slots of tile `index` < total.
  __device__ __forceinline__ void find(int index, int bn, int* expert, int* first, int* end) const {
    const int src = __builtin_ctzll(__ballot(index < upto));
    int left = index - (upto - tiles), e = 0, a = 0, b = 0;
#pragma unroll
    for (int i = 1; i <= 8; ++i) {
      const int n = (at[i] - at[i - 1] + bn - 1) / bn;
      if (left >= 0 && left < n) {
        e = 8 * static_cast<int>(threadIdx.x & 63) + i - 1;
        a = at[i - 1] + left * bn;
        b = at[i];
      }
      left -= n;
    }
    *expert = __builtin_amdgcn_readlane(e, src);
    *first = __builtin_amdgcn_readlane(a, src);
    const int stop = __builtin_amdgcn_readlane(b, src);
    *end = *first + bn < stop ? *first + bn : stop;
  }
};

// Lets a kernel use its dynamic LDS, once a device.
class LdsAllowance {
 public:
  int ask(const void* kernel, int bytes) {
    int dev = 0;
    QZ_HIP(hipGetDevice(&dev));
    if (dev > 63 || !(allowed_.load(std::memory_order_relaxed) >> dev & 1)) {
      QZ_HIP(hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes));
      if (dev <= 63) allowed_.fetch_or(uint64_t{1} << dev, std::memory_order_relaxed);
    }
    return QZ_OK;
  }

 private:
  std::atomic<uint64_t> allowed_{0};
};

// Token tiles of an expert layer, at most.
inline int64_t most_tiles(const I8Product& p, int bn) {
  return p.n / bn + (p.n < p.E ? p.n : p.E);
}

}  // namespace qz
