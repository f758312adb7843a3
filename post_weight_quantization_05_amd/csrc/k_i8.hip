// 8-bit integer storage: rows quantized to int8 with one scale each, and the solvers' unsigned codes
// to and from it.
#include <type_traits>

#include "i8_group.h"

namespace qz {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// TPR threads a row, CH chunks of eight elements each, which stay in registers between the row's
// maximum and its codes: one pass over X.  Rows up to 2048 columns take a wavefront and no barrier, where there
// are enough of them.  Past 32768 columns (eight chunks of 1024 threads) 128 registers a thread do not hold the row, the
// next one and the factors: the compiler keeps part of them in scratch, 20 to 152 bytes a thread and with factors 280 to
// 416 (16 to 20 bytes in fp32 with factors from 16385 columns on), and 2048 x 65536 bf16 takes 125 us (3.2 TB/s),
// with factors 248, fp32 241 and 361.
// A workgroup goes through several rows: the next one is on its way while one is worked on, and the
// column factors are loaded once.
//
// Bound by HBM: 8192 x 5120 bf16 with factors and values, 84 MB read and 126 written, 38 us a call in a
// warm loop (5.6 TB/s; torch's copy of 1 GiB reaches 5.1); 25600 x 5120 fp32 with values, 1.18 GB, 206 us
// (5.7 TB/s).  Few rows are bound by one row's chain, load, maximum, codes: 70 x 200 fp32 3.0 us, 13 x 12288
// bf16 4.0, most of it the launch.  Values leave past the caches in whole lines (42 -> 40 us in the former),
// and the quotients of a code take one multiplication unless they lie next to a half (i8_quant.h).
//
// GROUP: the first g.E workgroups sort an expert layer's pairs beside it.
template <int WT, bool VEC, bool FACTORS, bool GROUP, int TPR, int CH>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void i8_quantize_kernel(
    const void* __restrict__ X, int64_t rows, int64_t cols, int64_t ldx,
    const float* __restrict__ colf, int8_t* __restrict__ codes, float* __restrict__ scales,
    int32_t* __restrict__ sums, void* __restrict__ values, const Grouping g) {
  if constexpr (GROUP) {
    if (static_cast<int>(blockIdx.x) < g.E) {
      group_expert<(TPR < 256 ? 4 : TPR / 64)>(g, blockIdx.x);
      return;
    }
  }
  constexpr int kWaves = TPR / 64, kRows = TPR == 64 ? 4 : 1;   // rows of a workgroup at a time
  __shared__ uint32_t tops[2][kWaves];
  __shared__ int parts[2][kWaves];
  const int t = threadIdx.x % TPR, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int skip = GROUP ? g.E : 0;
  const int64_t P = i8_pitch(cols), step = static_cast<int64_t>(gridDim.x - skip) * kRows;
  int64_t row = (blockIdx.x - skip) * (int64_t)kRows + (TPR == 64 ? wave : 0);
  if (row >= rows) return;
  // Chunk c of this thread: eight neighbours, or in fp32 (VEC) four of them and four 4 TPR further on, so that
  // a wavefront's 16 bytes a lane are whole lines.
  constexpr bool kApart = VEC && WT == QZ_F32;
  constexpr int kSecond = kApart ? 4 * TPR : 4;
  auto place = [&](int c) { return static_cast<int64_t>(c * TPR * 8 + (kApart ? 4 : 8) * t); };
  auto load_f32 = [&](const void* p, int64_t at, int64_t c) {
    Raw8<QZ_F32> r;
    if constexpr (kApart) {
      const uint4 *a = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at + c),
                  *b = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at + c + kSecond);
      r.w[0] = c < cols ? *a : make_uint4(0, 0, 0, 0);
      r.w[1] = c + kSecond < cols ? *b : make_uint4(0, 0, 0, 0);
    } else {
      r = load8<QZ_F32, VEC>(p, at + c, cols - c);
    }
    return r;
  };
  float f[FACTORS ? CH : 1][8];
  if constexpr (FACTORS) {
#pragma unroll
    for (int c = 0; c < CH; ++c) numbers8(load_f32(colf, 0, place(c)), f[c]);
  }
  Raw8<WT> raw[CH];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if constexpr (WT == QZ_F32)
        raw[c] = load_f32(X, r * ldx, place(c));
      else
        raw[c] = load8<WT, VEC>(X, r * ldx + place(c), cols - place(c));
    }
  };
  load(row);
  for (int turn = 0; row < rows; row += step, turn ^= 1) {
    float v[CH][8];
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      numbers8(raw[c], v[c]);
      if constexpr (FACTORS) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] *= f[c][i];
      }
      top = top8(v[c], top);
    }
    if (row + step < rows) load(row + step);
    top = wave_top(top);
    if constexpr (kWaves > 1) {
      if (lane == 0) tops[turn][wave] = top;
      __syncthreads();   // the other buffer is free when the next row's barrier is passed
      top = wave_top(lane < kWaves ? tops[turn][lane] : 0u);
    }
    const RowScale sc = row_scale(top);
    int sum = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t at = place(c);
      if (at >= P) continue;
      float q[8];
      const uint2 w = codes8(v[c], sc, q);
      sum = add_codes(w.x, add_codes(w.y, sum));   // (zeros past the columns)
      int8_t* const to = codes + row * P + at;
      if constexpr (kApart) {
        *reinterpret_cast<uint32_t*>(to) = w.x;
        if (at + kSecond < P) *reinterpret_cast<uint32_t*>(to + kSecond) = w.y;
      } else {
        *reinterpret_cast<uint2*>(to) = w;
      }
      if (!values || at >= cols) continue;
      const int64_t o = row * cols + at;
      if constexpr (VEC) {   // written past the caches: nothing here reads them again
        if constexpr (WT == QZ_BF16) {
          u32x4 u;
#pragma unroll
          for (int i = 0; i < 4; ++i) u[i] = bf16_pair(q[2 * i] * sc.s, q[2 * i + 1] * sc.s);
          __builtin_nontemporal_store(u, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(values) + o));
        } else {
          float* const d = static_cast<float*>(values) + o;
          __builtin_nontemporal_store(f32x4{q[0] * sc.s, q[1] * sc.s, q[2] * sc.s, q[3] * sc.s}, reinterpret_cast<f32x4*>(d));
          if (at + kSecond < cols)
            __builtin_nontemporal_store(f32x4{q[4] * sc.s, q[5] * sc.s, q[6] * sc.s, q[7] * sc.s}, reinterpret_cast<f32x4*>(d + kSecond));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (at + i < cols) {
            if constexpr (WT == QZ_BF16)
              static_cast<uint16_t*>(values)[o + i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(q[i] * sc.s));
            else
              static_cast<float*>(values)[o + i] = q[i] * sc.s;
          }
      }
    }
    if (sums) {
      sum = wave_sum(sum);
      if constexpr (kWaves > 1) {
        if (lane == 0) parts[turn][wave] = sum;
        __syncthreads();
        sum = wave_sum(lane < kWaves ? parts[turn][lane] : 0);
      }
      if (t == 0) sums[row] = sum;
    }
    if (t == 0) scales[row] = sc.s;
  }
}

// A byte a thread at a time, with its place's division: 4096 x 12288 59 us either way (1.7 TB/s of 101 MB).  They stand
// between a solver and its product, once a layer.
__global__ __launch_bounds__(256) void i8_pack_kernel(const uint8_t* __restrict__ in, int64_t rows,
                                                      int64_t cols, int8_t* __restrict__ out) {
  const int64_t P = i8_pitch(cols);
  for (int64_t t = blockIdx.x * (int64_t)256 + threadIdx.x; t < rows * P; t += (int64_t)gridDim.x * 256) {
    const int64_t r = t / P, c = t % P;
    out[t] = c < cols ? static_cast<int8_t>(in[r * cols + c] ^ 0x80) : static_cast<int8_t>(0);
  }
}

__global__ __launch_bounds__(256) void i8_unpack_kernel(const int8_t* __restrict__ in, int64_t rows,
                                                        int64_t cols, uint8_t* __restrict__ out) {
  const int64_t P = i8_pitch(cols);
  for (int64_t t = blockIdx.x * (int64_t)256 + threadIdx.x; t < rows * cols; t += (int64_t)gridDim.x * 256) {
    const int64_t r = t / cols, c = t % cols;
    out[t] = static_cast<uint8_t>(in[r * P + c]) ^ 0x80;
  }
}

unsigned grid_for(int64_t items) {
  const int64_t b = ceil_div(items, 256);
  return static_cast<unsigned>(b < 65536 ? b : 65536);
}

}  // namespace

namespace {

template <bool GROUP>
int quantize(const void* X, int xt, int64_t rows, int64_t cols, int64_t ldx, const float* colf, int8_t* codes,
             float* scales, int32_t* sums, void* values, const Grouping& g, hipStream_t s) {
  // With factors, or in bf16, where a row is few bytes a thread, workgroups that fill the chip once and go
  // through the rows (8192 x 5120 bf16 with factors and values 41 us, a row each 52); else a row each
  // (25600 x 5120 fp32 with values 208 us, going through the rows 230).
  const bool through = colf || xt == QZ_BF16;
  auto go = [&](auto kernel, int tpr) {
    const int64_t groups = tpr == 64 ? ceil_div(rows, 4) : rows;
    const int64_t most = through ? 256 * (tpr < 256 ? 8 : 2048 / tpr) : int64_t{1} << 20;   // a launch's limit
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>((groups < most ? groups : most) + (GROUP ? g.E : 0))),
                       dim3(tpr < 256 ? 256 : tpr), 0, s, X, rows, cols, ldx, colf, codes, scales, sums, values, g);
    return check_launch("i8_quantize");
  };
  auto by_size = [&](auto type, auto vec, auto factors) {
    constexpr int WT = decltype(type)::value;
    constexpr bool VEC = decltype(vec)::value, F = decltype(factors)::value;
    if (cols <= 512) return go(i8_quantize_kernel<WT, VEC, F, GROUP, 64, 1>, 64);
    // few rows: a row's latency counts (300 rows of 2048 bf16, with the pairs sorted, 3.8 us against 6.6)
    if (cols <= 2048 && rows <= 1024) return go(i8_quantize_kernel<WT, VEC, F, GROUP, 256, 1>, 256);
    if (cols <= 1024) return go(i8_quantize_kernel<WT, VEC, F, GROUP, 64, 2>, 64);
    if (cols <= 2048) return go(i8_quantize_kernel<WT, VEC, F, GROUP, 64, 4>, 64);
    if (cols <= 4096) return go(i8_quantize_kernel<WT, VEC, F, GROUP, 256, 2>, 256);
    if (cols <= 6144) return go(i8_quantize_kernel<WT, VEC, F, GROUP, 256, 3>, 256);
    if (cols <= 8192) return go(i8_quantize_kernel<WT, VEC, F, GROUP, 256, 4>, 256);
    if (cols <= 16384) return go(i8_quantize_kernel<WT, VEC, F, GROUP, 1024, 2>, 1024);
    if (cols <= 32768) return go(i8_quantize_kernel<WT, VEC, F, GROUP, 1024, 4>, 1024);
    return go(i8_quantize_kernel<WT, VEC, F, GROUP, 1024, 8>, 1024);
  };
  auto by_type = [&](auto type) {
    const size_t size = decltype(type)::value == QZ_BF16 ? 2 : 4;
    auto on16 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    const bool vec = cols % 8 == 0 && ldx * size % 16 == 0 && on16(X) && on16(values) && on16(colf);
    if constexpr (!GROUP)
      if (colf)
        return vec ? by_size(type, std::true_type{}, std::true_type{}) : by_size(type, std::false_type{}, std::true_type{});
    return vec ? by_size(type, std::true_type{}, std::false_type{}) : by_size(type, std::false_type{}, std::false_type{});
  };
  return xt == QZ_BF16 ? by_type(std::integral_constant<int, QZ_BF16>{})
                       : by_type(std::integral_constant<int, QZ_F32>{});
}

}  // namespace

int launch_i8_quantize(const void* X, int xt, int64_t rows, int64_t cols, int64_t ldx,
                       const float* colf, int8_t* codes, float* scales, int32_t* sums, void* values,
                       hipStream_t s) {
  if (rows == 0) return QZ_OK;
  return quantize<false>(X, xt, rows, cols, ldx, colf, codes, scales, sums, values, Grouping{}, s);
}

int launch_i8_quantize_group(const void* X, int xt, int64_t rows, int64_t cols, int64_t ldx, int8_t* codes,
                             float* scales, int32_t* sums, const int32_t* ids, int k, int E, int32_t* offsets,
                             int32_t* order, hipStream_t s) {
  return quantize<true>(X, xt, rows, cols, ldx, nullptr, codes, scales, sums, nullptr,
                        Grouping{ids, rows * k, E, offsets, order}, s);
}

int launch_i8_pack(const uint8_t* codes, int64_t rows, int64_t cols, int8_t* out, hipStream_t s) {
  hipLaunchKernelGGL(i8_pack_kernel, dim3(grid_for(rows * i8_pitch(cols))), dim3(256), 0, s, codes, rows, cols, out);
  return check_launch("i8_pack");
}

int launch_i8_unpack(const int8_t* codes, int64_t rows, int64_t cols, uint8_t* out, hipStream_t s) {
  hipLaunchKernelGGL(i8_unpack_kernel, dim3(grid_for(rows * cols)), dim3(256), 0, s, codes, rows, cols, out);
  return check_launch("i8_unpack");
}

}  // namespace qz
