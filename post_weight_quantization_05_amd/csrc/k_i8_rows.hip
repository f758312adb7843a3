// Products of 8-bit integer rows with very few tokens: rows of W against one to four tokens, or
// against the experts' tokens one pair (token, r) at a time, by four-way dot products.  The tokens are
// quantized in the same launch where they come as numbers.
//
// Bound by the reading of W and, on small layers, by the launch and one chain: load a token, its maximum,
// codes, products, sums.  Every workgroup quantizes the tokens again (from L2; a second launch would cost
// 3 us more), while its first two blocks of W are on their way.  W goes straight to registers: no
// wavefront shares a row.  One token: 4096 -> 1024 4.1 us; 8 of 128 experts of 1024, d 4096, gate and up (67 MB)
// 16.3 us (4.1 TB/s with the launch), down (34 MB) 11.3.
#include <type_traits>

#include "i8_gemm.h"

namespace qz {

namespace {

constexpr int kCodes = -1;   // tokens that come as codes
constexpr int kRowsThreads = 256;

// What the tokens of a workgroup become in LDS: codes [rows][P rounded up to 1024], zero behind the
// columns, and each row's scale and sum of codes.
struct Staged {
  uint8_t* codes;
  float* scale;
  int* sum;
  int pitch;
};

// The first two chunks of eight elements that a thread has of a row (and their factors).  A wavefront's loads
// come back in the order of their issue, so these go out before the first blocks of W.
template <int QT>
struct RowStart {
  Raw8<QT> x[2];
  Raw8<QZ_F32> f[2];
};
// Of a row by the T threads t = 0 .. T - 1 of a wavefront or (T = kRowsThreads) of the workgroup.
template <int QT, bool VEC, bool FACTORS, int T>
__device__ __forceinline__ void fetch_row(const I8Product& p, int64_t row, int t, RowStart<QT>& r) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t c = 8 * (i * T + t);
    r.x[i] = load8<QT, VEC>(p.raw, row * p.ldraw + c, p.cols - c);
    if (FACTORS && p.colf) r.f[i] = load8<QZ_F32, VEC>(p.colf, c, p.cols - c);
  }
}
// start: null where it costs more registers than it gives (the row is loaded twice then, the second time from
// the caches).
template <int QT, bool VEC, bool FACTORS, int T>
__device__ __forceinline__ void stage_row(const I8Product& p, int64_t row, int i, int t, const Staged& s,
                                          uint32_t* tops, const RowStart<QT>* start) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t top = 0;
  auto with_factors = [&](const Raw8<QZ_F32>& raw, float (&v)[8]) {
    float f[8];
    numbers8(raw, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= f[j];
  };
  auto elements = [&](int c, float (&v)[8]) {
    numbers8(load8<QT, VEC>(p.raw, row * p.ldraw + c, p.cols - c), v);
    if (FACTORS && p.colf) with_factors(load8<QZ_F32, VEC>(p.colf, c, p.cols - c), v);
  };
  const int from = start ? 2 * T + t : t;
  float first[2][8];
  if (start) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      numbers8(start->x[j], first[j]);
      if (FACTORS && p.colf) with_factors(start->f[j], first[j]);
      top = top8(first[j], top);
    }
  }
  for (int c = 8 * from; c < p.cols; c += 8 * T) {
    float v[8];
    elements(c, v);
    top = top8(v, top);
  }
  top = wave_top(top);
  if constexpr (T > 64) {
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
    __syncthreads();   // before the next row's
  }
  const RowScale sc = row_scale(top);
  int sum = 0;
  auto write = [&](int c, const float (&v)[8]) {
    uint2 w = make_uint2(0, 0);
    if (c < p.cols) {
      float q[8];
      w = codes8(v, sc, q);
      sum = add_codes(w.x, add_codes(w.y, sum));
    }
    *reinterpret_cast<uint2*>(s.codes + i * s.pitch + c) = w;
  };
  if (start) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (8 * (j * T + t) < s.pitch) write(8 * (j * T + t), first[j]);
  }
  for (int c = 8 * from; c < s.pitch; c += 8 * T) {
    float v[8];
    elements(c, v);
    write(c, v);
  }
  if (p.zeros) {
    sum = wave_sum(sum);
    if constexpr (T > 64) {
      if (lane == 0) tops[wave] = static_cast<uint32_t>(sum);
      __syncthreads();
      sum = static_cast<int>(tops[0] + tops[1] + tops[2] + tops[3]);
      __syncthreads();
    }
  }
  if (t == 0) {
    s.scale[i] = sc.s;
    s.sum[i] = sum;
  }
}

// Rows first .. first + n - 1 of the tokens; all threads of the workgroup call it.  Up to three rows by the whole
// workgroup, with a few barriers each; more, a wavefront a row.
constexpr int kTogether = 3;
template <int QT, bool VEC, bool FACTORS>
__device__ __forceinline__ void fetch_rows(const I8Product& p, int64_t first, int n, RowStart<QT>& start) {
  const int tid = threadIdx.x;
  if (n <= kTogether)
    fetch_row<QT, VEC, FACTORS, kRowsThreads>(p, first, tid, start);
  else
    fetch_row<QT, VEC, FACTORS, 64>(p, first + (tid / 64 < n ? tid / 64 : 0), tid & 63, start);
}
template <int QT, bool VEC, bool FACTORS>
__device__ __forceinline__ void stage_rows(const I8Product& p, int64_t first, int n, const Staged& s, uint32_t* tops,
                                           const RowStart<QT>* start) {
  const int tid = threadIdx.x;
  if (n <= kTogether) {
    for (int i = 0; i < n; ++i)
      stage_row<QT, VEC, FACTORS, kRowsThreads>(p, first + i, i, tid, s, tops, i ? nullptr : start);
  } else {
    for (int i = tid / 64; i < n; i += kRowsThreads / 64)
      stage_row<QT, VEC, FACTORS, 64>(p, first + i, i, tid & 63, s, tops, i < kRowsThreads / 64 ? start : nullptr);
  }
  __syncthreads();
}
// Rows that come as codes: 16 bytes a thread at a time, the first of them fetched before.
__device__ __forceinline__ uint4 code_piece(const I8Product& p, int64_t first, int n, const Staged& s, int c) {
  const int i = c / s.pitch, at = c % s.pitch;
  return c < n * s.pitch && at < p.P ? *reinterpret_cast<const uint4*>(p.X + (first + i) * p.P + at) : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ void stage_codes(const I8Product& p, int64_t first, int n, const Staged& s, const uint4& start) {
  const int tid = threadIdx.x;
  for (int c = 16 * tid; c < n * s.pitch; c += 16 * kRowsThreads)
    *reinterpret_cast<uint4*>(s.codes + c) = c == 16 * tid ? start : code_piece(p, first, n, s, c);
  if (tid < n) {
    s.scale[tid] = p.sx[first + tid];
    s.sum[tid] = p.zeros ? p.xsum[first + tid] : 0;
  }
  __syncthreads();
}

// A wavefront has R rows of W (kGateUp: R / 2 gate rows and their up rows); N tokens for kPlain.
// Lane l has 16 bytes of every 1024 columns; blocks of U times 1024 columns of R rows are loaded two
// ahead, the first two before the tokens are staged.
template <Form FORM, int QT, bool VEC, int N, int R>
__global__ __launch_bounds__(kRowsThreads) void i8_rows_kernel(const I8Product p) {
  constexpr int U = R >= 8 ? 1 : 8 / R;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float xscale[N];
  __shared__ int xsums[N];
  __shared__ uint32_t tops[4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int kOut = FORM == kGateUp ? R / 2 : R;   // results of a wavefront (for each token)
  const int64_t r0 = (blockIdx.x * (int64_t)4 + wave) * kOut;
  const int pair = FORM == kGateUp ? blockIdx.y : 0;
  const uint32_t P = static_cast<uint32_t>(p.P);
  const Staged s{smem, xscale, xsums, static_cast<int>(round_up(p.P, 1024))};

  const int expert = FORM == kGateUp ? p.ids[pair] : 0;
  if (FORM == kGateUp && (expert < 0 || expert >= p.E)) return;   // nobody reads its hidden row
  const int64_t w_row0 = expert * (FORM == kGateUp ? 2 : 1) * p.d_o;
  auto row_of = [&](int i) {   // of the expert's
    const int64_t r = r0 + (FORM == kGateUp ? i % kOut : i);
    return (r < p.d_o ? r : p.d_o - 1) + (FORM == kGateUp && i >= kOut ? p.d_o : 0);
  };
  const int blocks = (s.pitch / 1024 + U - 1) / U;
  auto load = [&](int b, i32x4 (&w)[R][U]) {
    if (b >= blocks) return;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int8_t* row = p.W + (w_row0 + row_of(i)) * p.P;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t c = static_cast<uint32_t>(b * U + u) * 1024 + 16 * lane;
        w[i][u] = *reinterpret_cast<const i32x4*>(row + (c < P ? c : 0));   // past the row: against zeros
      }
    }
  };
  int acc[R][N];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int t = 0; t < N; ++t) acc[i][t] = 0;
  auto use = [&](int b, const i32x4 (&w)[R][U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = (b * U + u) * 1024 + 16 * lane;
      if (U > 1 && c >= s.pitch) continue;
#pragma unroll
      for (int t = 0; t < N; ++t) {
        const i32x4 x = *reinterpret_cast<const i32x4*>(s.codes + t * s.pitch + c);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][t] = __builtin_amdgcn_sdot4(w[i][u][j], x[j], acc[i][t], false);
      }
    }
  };
  i32x4 even[R][U], odd[R][U];
  const int64_t first = FORM == kGateUp ? pair / p.k : 0;
  std::conditional_t<QT == kCodes, uint4, RowStart<QT == kCodes ? QZ_F32 : QT>> start;
  if constexpr (QT == kCodes)
    start = code_piece(p, first, N, s, 16 * threadIdx.x);
  else
    fetch_rows<QT, VEC, FORM == kPlain>(p, first, N, start);
  __builtin_amdgcn_sched_barrier(0);
  load(0, even);
  load(1, odd);
  // What the lane's result is made with, on its way as early: of row lane / N (kGateUp: lane).
  const int at = lane < R * N ? lane / N : 0;
  const int64_t my_row = w_row0 + row_of(at);
  const float my_sw = p.sw[my_row];
  const int my_shift = p.zeros ? p.zeros[my_row] - 128 : 0;
  const float my_bias = FORM == kPlain && p.bias ? p.bias[my_row] : 0.f;
  if constexpr (QT == kCodes)
    stage_codes(p, first, N, s, start);
  else
    stage_rows<QT, VEC, FORM == kPlain>(p, first, N, s, tops, &start);
  for (int b = 0; b < blocks; b += 2) {
    use(b, even);
    load(b + 2, even);
    if (b + 1 >= blocks) break;
    use(b + 1, odd);
    load(b + 3, odd);
  }
  // Lane l's sum of row i and token t, l = i N + t.
  int a = 0;
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int t = 0; t < N; ++t) {
      const int total = wave_sum(acc[i][t]);
      a = lane == i * N + t ? total : a;
    }
  if constexpr (FORM == kGateUp) {
    const float v = scaled(a, my_shift, xsums[0], xscale[0], my_sw, 0.f);
    const float up = __shfl(v, lane + kOut);
    if (lane < kOut && r0 + lane < p.d_o) static_cast<float*>(p.Y)[pair * p.ldy + r0 + lane] = silu(v) * up;
  } else {
    const int t = lane % N;
    const int64_t r = r0 + lane / N;
    if (lane < R * N && r < p.d_o) {
      const float v = scaled(a, my_shift, xsums[t], xscale[t], my_sw, my_bias);
      if (p.yt == QZ_BF16)
        static_cast<uint16_t*>(p.Y)[t * p.ldy + r] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
      else
        static_cast<float*>(p.Y)[t * p.ldy + r] = v;
    }
  }
}

// The down products of a token's pairs and their weighted sum.  SPLIT wavefronts share the pairs (wavefront
// w has w % SPLIT, w % SPLIT + SPLIT, ...), and 4 / SPLIT of them the rows of W, R each; the first two
// blocks of W are on their way before the hidden rows are staged.
template <bool VEC, int SPLIT, int R>
__global__ __launch_bounds__(kRowsThreads) void i8_rows_down_kernel(const I8Product p) {
  constexpr int kOut = R * (4 / SPLIT);
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float xscale[QZ_ROUTE_MAX_TOP_K];
  __shared__ int part[QZ_ROUTE_MAX_TOP_K][kOut];   // sums, and then the weighted results' bits
  __shared__ int xsums[QZ_ROUTE_MAX_TOP_K];
  __shared__ uint32_t tops[4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), turn = wave % SPLIT;
  const int64_t wg0 = blockIdx.x * (int64_t)kOut, r0 = wg0 + wave / SPLIT * R;
  const int64_t pair0 = blockIdx.y * (int64_t)p.k;
  const uint32_t P = static_cast<uint32_t>(p.P);
  const Staged s{smem, xscale, xsums, static_cast<int>(round_up(p.P, 1024))};
  const int per = s.pitch / 1024, mine = (p.k - turn + SPLIT - 1) / SPLIT, blocks = mine * per;   // of this wavefront
  auto expert_of = [&](int at) {   // -1: not here
    const int e = p.ids[pair0 + at];
    return e >= 0 && e < p.E ? e : -1;
  };
  auto load = [&](int b, i32x4 (&w)[R]) {
    if (b >= blocks) return;
    int e = expert_of(turn + SPLIT * (b / per));
    if (e < 0) e = 0;
    const uint32_t c = static_cast<uint32_t>(b % per) * 1024 + 16 * lane, at = c < P ? c : 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t r = e * p.d_o + (r0 + i < p.d_o ? r0 + i : p.d_o - 1);
      w[i] = *reinterpret_cast<const i32x4*>(p.W + r * p.P + at);
    }
  };
  int acc[R];
#pragma unroll
  for (int i = 0; i < R; ++i) acc[i] = 0;
  auto use = [&](int b, const i32x4 (&w)[R]) {
    const int at = turn + SPLIT * (b / per);
    const i32x4 x = *reinterpret_cast<const i32x4*>(s.codes + at * s.pitch + b % per * 1024 + 16 * lane);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i] = __builtin_amdgcn_sdot4(w[i][j], x[j], acc[i], false);
    if ((b + 1) % per) return;
    int a = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {   // a pair's sums
      const int total = wave_sum(acc[i]);
      a = lane == i ? total : a;
      acc[i] = 0;
    }
    if (lane < R) part[at][r0 - wg0 + lane] = a;
  };
  i32x4 even[R], odd[R];
  RowStart<QZ_F32> start;
  if constexpr (SPLIT == 4) {   // of the wavefront's first pair (with more workgroups a compute unit, the registers cost more)
    fetch_row<QZ_F32, VEC, false, 64>(p, pair0 + (wave < p.k ? wave : 0), lane, start);
    __builtin_amdgcn_sched_barrier(0);
  }
  load(0, even);
  load(1, odd);
  // What a pair's result of a row is made with, on its way as early: a thread has up to kEach of them.
  constexpr int kEach = QZ_ROUTE_MAX_TOP_K * kOut / kRowsThreads;
  float my_sw[kEach], my_weight[kEach];
  int my_shift[kEach];
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int i = (j * kRowsThreads + threadIdx.x) / kOut, o = threadIdx.x % kOut;
    const int e = i < p.k ? expert_of(i) : -1;
    my_sw[j] = my_weight[j] = 0.f;
    my_shift[j] = 0;
    if (e >= 0) {
      const int64_t r = e * p.d_o + (wg0 + o < p.d_o ? wg0 + o : p.d_o - 1);
      my_sw[j] = p.sw[r];
      my_weight[j] = p.pair_weight[pair0 + i];
      if (p.zeros) my_shift[j] = p.zeros[r] - 128;
    }
  }
  if constexpr (SPLIT == 4) {   // each wavefront its own: its LDS accesses stay in order, the compiler's too
    for (int i = wave; i < p.k; i += 4) {
      if (i >= 4) fetch_row<QZ_F32, VEC, false, 64>(p, pair0 + i, lane, start);
      stage_row<QZ_F32, VEC, false, 64>(p, pair0 + i, i, lane, s, nullptr, &start);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  } else {
    stage_rows<QZ_F32, VEC, false>(p, pair0, p.k, s, tops, nullptr);
  }
  for (int b = 0; b < blocks; b += 2) {
    use(b, even);
    load(b + 2, even);
    if (b + 1 >= blocks) break;
    use(b + 1, odd);
    load(b + 3, odd);
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int i = (j * kRowsThreads + threadIdx.x) / kOut, o = threadIdx.x % kOut;
    if (i < p.k)
      part[i][o] = __float_as_int(my_weight[j] * scaled(part[i][o], my_shift[j], xsums[i], xscale[i], my_sw[j], 0.f));
  }
  __syncthreads();
  const int64_t r = wg0 + threadIdx.x;
  if (threadIdx.x < kOut && r < p.d_o) {
    float y = 0.f;
    for (int i = 0; i < p.k; ++i)
      if (expert_of(i) >= 0) y += __int_as_float(part[i][threadIdx.x]);
    static_cast<uint16_t*>(p.Y)[blockIdx.y * p.ldy + r] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(y));
  }
}

template <Form FORM, int QT, bool VEC, int N, int R>
int launch_rows(const I8Product& p, int64_t y, hipStream_t s) {
  constexpr int kOut = 4 * (FORM == kGateUp ? R / 2 : R);
  hipLaunchKernelGGL((i8_rows_kernel<FORM, QT, VEC, N, R>), dim3(static_cast<unsigned>(ceil_div(p.d_o, kOut)), static_cast<unsigned>(y)),
                     dim3(kRowsThreads), static_cast<size_t>(N * round_up(p.P, 1024)), s, p);
  return check_launch("i8_rows");
}

template <Form FORM, int QT, bool VEC>
int by_tokens(const I8Product& p, int64_t y, hipStream_t s) {
  if constexpr (FORM == kGateUp) {
    return launch_rows<FORM, QT, VEC, 1, 8>(p, y, s);
  } else {
    // rows a wavefront: enough wavefronts for the chip first
    auto by_rows = [&](auto n) {
      constexpr int N = decltype(n)::value;
      if (p.d_o <= 2048) return launch_rows<FORM, QT, VEC, N, 1>(p, 1, s);
      if (p.d_o <= 8192) return launch_rows<FORM, QT, VEC, N, 4>(p, 1, s);
      return launch_rows<FORM, QT, VEC, N, 8>(p, 1, s);
    };
    switch (p.n) {
      case 1: return by_rows(std::integral_constant<int, 1>{});
      case 2: return by_rows(std::integral_constant<int, 2>{});
      case 3: return by_rows(std::integral_constant<int, 3>{});
      default: return by_rows(std::integral_constant<int, 4>{});
    }
  }
}

// Whether the tokens' rows (and the factors) are whole chunks of eight on 16-byte boundaries.
bool vector_rows(const I8Product& p) {
  const size_t size = p.rt == QZ_BF16 ? 2 : 4;
  auto on16 = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
  return p.cols % 8 == 0 && p.ldraw * size % 16 == 0 && on16(p.raw) && on16(p.colf);
}

template <Form FORM>
int by_type(const I8Product& p, int64_t y, hipStream_t s) {
  if constexpr (FORM == kPlain)
    if (!p.raw) return by_tokens<FORM, kCodes, true>(p, y, s);
  const bool vec = vector_rows(p);
  if (p.rt == QZ_BF16)
    return vec ? by_tokens<FORM, QZ_BF16, true>(p, y, s) : by_tokens<FORM, QZ_BF16, false>(p, y, s);
  return vec ? by_tokens<FORM, QZ_F32, true>(p, y, s) : by_tokens<FORM, QZ_F32, false>(p, y, s);
}

}  // namespace

int launch_i8_rows(const I8Product& p, hipStream_t s) { return by_type<kPlain>(p, 1, s); }
int launch_i8_rows_gate_up(const I8Product& p, hipStream_t s) { return by_type<kGateUp>(p, p.n, s); }
int launch_i8_rows_down(const I8Product& p, int64_t tokens, hipStream_t s) {
  auto go = [&](auto kernel, int rows) {
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(ceil_div(p.d_o, rows)), static_cast<unsigned>(tokens)),
                       dim3(kRowsThreads), static_cast<size_t>(p.k * round_up(p.P, 1024)), s, p);
    return check_launch("i8_rows_down");
  };
  // Few workgroups: as many wavefronts on a token's pairs as there are pairs for, so that there are more of
  // them (1 token 8 of 128 x 1024, d 4096: 12.3 us, half as many 18.8; now 11.3); else more rows for each staging
  // (4 tokens there: 28.8 us against 32.8, now 28.0; 7 tokens 2 of 8 x 2048: 17.2 against 20.9).
  const bool many = tokens * ceil_div(p.d_o, 16) >= 512;
  auto by_pairs = [&](auto vec) {
    constexpr bool VEC = decltype(vec)::value;
    if (p.k >= 4) return many ? go(i8_rows_down_kernel<VEC, 2, 16>, 32) : go(i8_rows_down_kernel<VEC, 4, 16>, 16);
    if (p.k >= 2 && !many) return go(i8_rows_down_kernel<VEC, 2, 8>, 16);
    return many ? go(i8_rows_down_kernel<VEC, 1, 8>, 32) : go(i8_rows_down_kernel<VEC, 1, 4>, 16);
  };
  return vector_rows(p) ? by_pairs(std::true_type{}) : by_pairs(std::false_type{});
}

}  // namespace qz
