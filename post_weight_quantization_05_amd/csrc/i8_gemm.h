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

// An integer sum with its zero point, scales and bias.  shift: the zero point less 128; |xsum| < 2^23, so
// the product takes the 24-bit multiplier.
__device__ __forceinline__ float scaled(int a, int shift, int xsum, float sx, float sw, float bias) {
  return fmaf(static_cast<float>(a - __mul24(shift, xsum)) * sx, sw, bias);
}

// g / (1 + e^-g) by the hardware's power of two and reciprocal, a last bit off each: g log2 e is off by half
// of one, so the whole by less than (4 + |g|) 2^-23 of itself.  (By the library's exponential and an exact
// quotient an expert layer's gate and up products spent a sixth of their time here.)
__device__ __forceinline__ float silu(float g) {
  return g * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * g));
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
