// Microscaled 4-bit (MX4) quantisation: round-to-nearest of a matrix on E2M1 elements with
// one power-of-two factor per 32 columns of a row.
//
// One pass over W, bound by HBM: 12288 x 4096 bf16 with values, 228 MB, 38.6 us (5.9 TB/s); 5120 x
// 25600 fp32 with values under column weights, 1.12 GB, 216 us (5.2 TB/s); a copy by the library
// reaches 4.9 TB/s of reads and writes together.  Four lanes a block, eight elements each in 16-byte
// accesses; the maximum and the 64-bit error sums pass between the four lanes.
#include <type_traits>

#include "mx4.h"

namespace qz {

namespace {

constexpr int kThreads = 256;

// Values of the other lanes of a quad (lane ^ 1, lane ^ 2), by data-parallel moves.
template <int X>
__device__ __forceinline__ uint32_t quad_xor(uint32_t v) {
  return __builtin_amdgcn_mov_dpp(v, X == 1 ? 0xB1 : 0x4E, 0xf, 0xf, true);
}
template <int X>
__device__ __forceinline__ double quad_xor(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint64_t lo = quad_xor<X>(static_cast<uint32_t>(u)), hi = quad_xor<X>(static_cast<uint32_t>(u >> 32));
  return __builtin_bit_cast(double, hi << 32 | lo);
}
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = quad_xor<1>(v);
  v = o > v ? o : v;
  o = quad_xor<2>(v);
  return o > v ? o : v;
}
__device__ __forceinline__ double quad_sum(double v) {
  v += quad_xor<1>(v);
  return v + quad_xor<2>(v);
}

typedef float f32x2 __attribute__((ext_vector_type(2)));

// Eight magnitudes rounded onto the factor, as eight codes; the factor is the exponent field of
// an fp32 word, and the conversion rounds to nearest even and saturates.
__device__ __forceinline__ uint32_t round8(const float (&v)[8], float factor) {
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], factor, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], factor, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], factor, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], factor, 3);
}
__device__ __forceinline__ void widen8(uint32_t q, float factor, float (&x)[8]) {
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, factor, 0);
  const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, factor, 1);
  const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, factor, 2);
  const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, factor, 3);
  x[0] = a[0]; x[1] = a[1]; x[2] = b[0]; x[3] = b[1];
  x[4] = c[0]; x[5] = c[1]; x[6] = d[0]; x[7] = d[1];
}

// Squared error of eight elements in 64 bits.  w - q is exact in fp32 (q is 0 or within a factor
// of two of w, or w saturates at less than twice the top), so only the sums round.
template <bool WEIGHTED>
__device__ __forceinline__ double error8(const float (&v)[8], const float (&x)[8],
                                         const float (&h)[8]) {
  double s = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double d = v[i] - x[i];
    s = WEIGHTED ? fma(d * d, static_cast<double>(h[i]), s) : fma(d, d, s);
  }
  return s;
}

// Four lanes per block, eight columns each: every load and store of a wavefront is contiguous
// (bf16: 16 bytes a lane), and the block's maximum and sums are two moves inside the quad.  The
// work is one pass over W, bound by HBM.  VEC: rows of W and of `values`, and colw, start on 16-byte
// boundaries and are whole chunks of eight; other rows go element by element.  Idx: 32-bit where
// the chunks' index fits, since its division is the longest computation of the FLOOR rule.
enum Rule { kFloor, kLeast, kLeastWeighted };

template <int WT, Rule RULE, bool VEC, class Idx>
__global__ __launch_bounds__(kThreads) void mx4_quantize_kernel(
    const void* __restrict__ W, int64_t rows, int64_t cols, int64_t ldw,
    const float* __restrict__ colw, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
    void* __restrict__ values) {
  const Idx per_row = static_cast<Idx>(mx_blocks(cols)) * 4;
  const Idx total = static_cast<Idx>(rows) * per_row;
  for (Idx t = static_cast<Idx>(blockIdx.x) * kThreads + threadIdx.x; t < total;
       t += static_cast<Idx>(gridDim.x) * kThreads) {
    const Idx r = t / per_row;
    const int64_t c0 = static_cast<int64_t>(t - r * per_row) * 8;
    const int64_t at = static_cast<int64_t>(r) * ldw + c0;
    const int64_t left = cols - c0;   // may be <= 0 in the last block
    float v[8];
    if constexpr (VEC) {
      if (left > 0) {
        if constexpr (WT == QZ_BF16) {
          const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(W) + at);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
          }
        } else {
          const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(W) + at);
          const f32x4 a = p[0], b = p[1];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < left ? load_w<WT>(W, at + i) : 0.f;
    }
    uint32_t top = 0;   // magnitudes compare as integers, and a NaN is above every number
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
      top = b > top ? b : top;
    }
    const uint32_t ex = quad_max(top) >> 23;
    uint32_t e = ex > 2 ? ex - 2 : 0;
    uint32_t q = round8(v, mx_factor(e));
    if constexpr (RULE != kFloor) {
      float h[8], x[8], y[8];
      if constexpr (RULE == kLeastWeighted) {
        if constexpr (VEC) {
          const f32x4* p = reinterpret_cast<const f32x4*>(colw + (left > 0 ? c0 : 0));
          const f32x4 a = p[0], b = p[1];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            h[i] = a[i];
            h[4 + i] = b[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) h[i] = i < left ? colw[c0 + i] : 0.f;
        }
      }
      const uint32_t q1 = round8(v, mx_factor(e + 1));
      widen8(q, mx_factor(e), x);
      widen8(q1, mx_factor(e + 1), y);
      const double d0 = quad_sum(error8<RULE == kLeastWeighted>(v, x, h));
      const double d1 = quad_sum(error8<RULE == kLeastWeighted>(v, y, h));
      if (d1 < d0) {   // the same in the four lanes: both sums add the same pairs
        q = q1;
        e += 1;
      }
    }
    if (ex == 255) {
      q = 0;
      e = 255;
    }
    *reinterpret_cast<uint32_t*>(codes + static_cast<int64_t>(t) * 4) = q;
    if ((t & 3) == 0) scales[t >> 2] = static_cast<uint8_t>(e);
    if (values && left > 0) {
      float x[8];
      widen8(q, mx_factor(e), x);
      const int64_t o = static_cast<int64_t>(r) * cols + c0;
      if constexpr (VEC) {
        if constexpr (WT == QZ_BF16) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)   // exact: the upper half of the fp32 value
            w[i] = __float_as_uint(x[2 * i]) >> 16 | (__float_as_uint(x[2 * i + 1]) & 0xffff0000u);
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(values) + o) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(values) + o);
          p[0] = f32x4{x[0], x[1], x[2], x[3]};
          p[1] = f32x4{x[4], x[5], x[6], x[7]};
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < left) {
            if constexpr (WT == QZ_BF16)
              static_cast<uint16_t*>(values)[o + i] = static_cast<uint16_t>(__float_as_uint(x[i]) >> 16);
            else
              static_cast<float*>(values)[o + i] = x[i];
          }
      }
    }
  }
}

// One thread per block: the codes as integers 2 x (E2M1 value) and the factor halved, which
// is qz_objective_i32's form of the same numbers (zero point 0).
__global__ __launch_bounds__(kThreads) void mx4_unpack_kernel(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows,
    int64_t cols, int32_t* __restrict__ out, float* __restrict__ out_scales,
    uint8_t* __restrict__ zeros) {
  const int64_t G = mx_blocks(cols);
  for (int64_t t = blockIdx.x * (int64_t)kThreads + threadIdx.x; t < rows * G;
       t += (int64_t)gridDim.x * kThreads) {
    const int64_t r = t / G, c0 = (t % G) * kMxBlock;
    const uint4 c = *reinterpret_cast<const uint4*>(codes + t * 16);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < kMxBlock; ++i) {
      const uint32_t q = (w[i / 8] >> (4 * (i % 8))) & 15u;
      // magnitude codes 0..7 -> 0 1 2 3 4 6 8 12, four bits each
      const int mag = static_cast<int>((0xC8643210u >> (4 * (q & 7u))) & 15u);
      if (c0 + i < cols) out[r * cols + c0 + i] = (q & 8u) ? -mag : mag;
    }
    const uint32_t e = scales[t];
    // 2^(e - 128): below e = 2 a subnormal number
    out_scales[t] = e == 255 ? __uint_as_float(0x7fc00000u)
                             : __uint_as_float(e >= 2 ? (e - 1) << 23 : 1u << (21 + e));
    zeros[t] = 0;
  }
}

int grid_for(int64_t items) {
  const int64_t b = ceil_div(items, kThreads);
  return static_cast<int>(b < (1 << 20) ? b : (1 << 20));
}

}  // namespace

namespace {

template <int WT, Rule RULE>
int quantize(const void* W, int64_t rows, int64_t cols, int64_t ldw, const float* colw,
             uint8_t* codes, uint8_t* scales, void* values, hipStream_t s) {
  const size_t size = WT == QZ_BF16 ? 2 : 4;
  auto on16 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  const bool vec = cols % 8 == 0 && ldw * size % 16 == 0 && on16(W) && on16(values) && on16(colw);
  const int64_t items = rows * mx_blocks(cols) * 4;
  const dim3 g(grid_for(items));
  // the grid's stride may carry the 32-bit index past the end once
  const bool narrow = items + int64_t{1} * g.x * kThreads < (int64_t{1} << 32);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, g, dim3(kThreads), 0, s, W, rows, cols, ldw, colw, codes, scales, values);
    return check_launch("mx4_quantize");
  };
  if (!narrow) return go(mx4_quantize_kernel<WT, RULE, false, uint64_t>);
  return vec ? go(mx4_quantize_kernel<WT, RULE, true, uint32_t>)
             : go(mx4_quantize_kernel<WT, RULE, false, uint32_t>);
}

}  // namespace

int launch_mx4_quantize(const void* W, int wt, int64_t rows, int64_t cols, int64_t ldw, int rule,
                        const float* colw, uint8_t* codes, uint8_t* scales, void* values,
                        hipStream_t s) {
  auto by_rule = [&](auto type) {
    constexpr int WT = decltype(type)::value;
    const auto f = rule != QZ_MX4_LEAST ? quantize<WT, kFloor>
                   : colw               ? quantize<WT, kLeastWeighted>
                                        : quantize<WT, kLeast>;
    return f(W, rows, cols, ldw, colw, codes, scales, values, s);
  };
  return wt == QZ_BF16 ? by_rule(std::integral_constant<int, QZ_BF16>{})
                       : by_rule(std::integral_constant<int, QZ_F32>{});
}

int launch_mx4_unpack(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                      int32_t* out, float* out_scales, uint8_t* zeros, hipStream_t s) {
  hipLaunchKernelGGL(mx4_unpack_kernel, dim3(grid_for(rows * mx_blocks(cols))), dim3(kThreads), 0,
                     s, codes, scales, rows, cols, out, out_scales, zeros);
  return check_launch("mx4_unpack");
}

}  // namespace qz
