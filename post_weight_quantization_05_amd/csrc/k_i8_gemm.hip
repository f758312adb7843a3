// Products of 8-bit integer rows: Y = X W^T with a scale per row of X and of W, plain or grouped by
// expert.
#include "qz_internal.h"

namespace qz {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

enum Form { kPlain, kGateUp, kDown };

// Expert and slots of the token tile `index` of `bn` slots; false past the last one.
__device__ __forceinline__ bool find_tile(const I8Product& p, int64_t index, int bn, int* expert,
                                          int64_t* first, int64_t* end) {
  for (int e = 0; e < p.E; ++e) {
    const int a = p.offsets[e], b = p.offsets[e + 1], tiles = (b - a + bn - 1) / bn;
    if (index < tiles) {
      *expert = e;
      *first = a + index * bn;
      *end = *first + bn < b ? *first + bn : b;
      return true;
    }
    index -= tiles;
  }
  return false;
}

__device__ __forceinline__ float scaled(int a, int xsum, int zero, float sx, float sw, float bias) {
  return fmaf(static_cast<float>(a - (zero - 128) * xsum) * sx, sw, bias);
}

// A wavefront per 16 rows of W by 16 rows of X, operands straight from memory.
template <Form FORM>
__global__ __launch_bounds__(64) void i8_product_kernel(const I8Product p) {
  const int lane = threadIdx.x, m = lane & 15, q = lane >> 4;
  int expert = 0;
  int64_t first = blockIdx.y * (int64_t)16, end = p.n;
  if constexpr (FORM != kPlain)
    if (!find_tile(p, blockIdx.y, 16, &expert, &first, &end)) return;
  const int64_t r0 = blockIdx.x * (int64_t)16;
  const int64_t w_rows = (FORM == kGateUp ? 2 : 1) * p.d_o, base = expert * w_rows;
  const int64_t wr = r0 + m < p.d_o ? r0 + m : p.d_o - 1;
  const int64_t slot = first + m < end ? first + m : end - 1;
  const int64_t pair = FORM == kPlain ? slot : p.order[slot];
  const int64_t xr = FORM == kGateUp ? pair / p.k : slot;
  const int8_t* w = p.W + (base + wr) * p.P + 16 * q;
  const int8_t* u = FORM == kGateUp ? w + p.d_o * p.P : w;
  const int8_t* x = p.X + xr * p.P + 16 * q;
  i32x4 acc = {0, 0, 0, 0}, acu = {0, 0, 0, 0};
  for (int64_t c = 0; c < p.P; c += 64) {
    const i32x4 xv = *reinterpret_cast<const i32x4*>(x + c);
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(*reinterpret_cast<const i32x4*>(w + c), xv, acc, 0, 0, 0);
    if constexpr (FORM == kGateUp)
      acu = __builtin_amdgcn_mfma_i32_16x16x64_i8(*reinterpret_cast<const i32x4*>(u + c), xv, acu, 0, 0, 0);
  }
  if (first + m >= end) return;
  const float sx = p.sx[xr];
  const int xsum = p.zeros ? p.xsum[xr] : 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + 4 * q + i;
    if (r >= p.d_o) continue;
    const int zero = p.zeros ? p.zeros[base + r] : 128;
    const float v = scaled(acc[i], xsum, zero, sx, p.sw[base + r], FORM == kPlain && p.bias ? p.bias[r] : 0.f);
    if constexpr (FORM == kPlain) {
      if (p.yt == QZ_BF16)
        static_cast<uint16_t*>(p.Y)[slot * p.ldy + r] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
      else
        static_cast<float*>(p.Y)[slot * p.ldy + r] = v;
    } else if constexpr (FORM == kGateUp) {
      const int64_t ru = base + p.d_o + r;
      const float up = scaled(acu[i], xsum, p.zeros ? p.zeros[ru] : 128, sx, p.sw[ru], 0.f);
      static_cast<float*>(p.Y)[slot * p.ldy + r] = v / (1.f + expf(-v)) * up;
    } else {
      static_cast<float*>(p.Y)[pair * p.ldy + r] = v * p.pair_weight[pair];
    }
  }
}

template <Form FORM>
int launch(const I8Product& p, hipStream_t s) {
  const int64_t tiles = FORM == kPlain ? ceil_div(p.n, 16) : ceil_div(p.n, 16) + (p.n < p.E ? p.n : p.E);
  for (int64_t t = 0; t < tiles; t += 65535) {   // a launch's limit
    if (FORM != kPlain && t > 0) return fail(QZ_EINVAL, "i8_moe: too many tokens");
    I8Product q = p;
    q.n = p.n - 16 * t;
    q.X = p.X + 16 * t * p.P;
    q.sx = p.sx + 16 * t;
    q.xsum = p.xsum ? p.xsum + 16 * t : nullptr;
    q.Y = static_cast<char*>(p.Y) + 16 * t * p.ldy * (p.yt == QZ_BF16 ? 2 : 4);
    const dim3 g(static_cast<unsigned>(ceil_div(p.d_o, 16)), static_cast<unsigned>(tiles - t < 65535 ? tiles - t : 65535));
    hipLaunchKernelGGL((i8_product_kernel<FORM>), g, dim3(64), 0, s, q);
    QZ_TRY(check_launch("i8_product"));
  }
  return QZ_OK;
}

}  // namespace

size_t i8_product_ws(int64_t, int64_t, int64_t) { return 0; }
int launch_i8_product(const I8Product& p, hipStream_t s) { return launch<kPlain>(p, s); }
int launch_i8_gate_up(const I8Product& p, hipStream_t s) { return launch<kGateUp>(p, s); }
int launch_i8_down(const I8Product& p, hipStream_t s) { return launch<kDown>(p, s); }

}  // namespace qz
