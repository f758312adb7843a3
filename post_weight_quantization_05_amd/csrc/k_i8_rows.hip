// Products of 8-bit integer rows with very few tokens: rows of W against one to four tokens, or
// against the experts' tokens one pair (token, r) at a time, by four-way dot products.  The tokens are
// quantized in the same launch where they come as numbers.
#include <type_traits>

#include "i8_gemm.h"

namespace qz {

namespace {

constexpr int kCodes = -1;   // tokens that come as codes
constexpr int kRowsThreads = 256;

// Sum over the wavefront, in every lane.
__device__ __forceinline__ int lanes_sum(int v) {
  v += __builtin_amdgcn_mov_dpp(v, 0xB1, 0xf, 0xf, true);    // lane ^ 1
  v += __builtin_amdgcn_mov_dpp(v, 0x4E, 0xf, 0xf, true);    // lane ^ 2
  v += __builtin_amdgcn_mov_dpp(v, 0x141, 0xf, 0xf, true);   // mirrored in eight
  v += __builtin_amdgcn_mov_dpp(v, 0x140, 0xf, 0xf, true);   // mirrored in sixteen
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = static_cast<int>(a[0]) + static_cast<int>(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return static_cast<int>(b[0]) + static_cast<int>(b[1]);
}
__device__ __forceinline__ uint32_t lanes_top(uint32_t v) {
  const auto up = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
  v = up(v, __builtin_amdgcn_mov_dpp(v, 0xB1, 0xf, 0xf, true));
  v = up(v, __builtin_amdgcn_mov_dpp(v, 0x4E, 0xf, 0xf, true));
  v = up(v, __builtin_amdgcn_mov_dpp(v, 0x141, 0xf, 0xf, true));
  v = up(v, __builtin_amdgcn_mov_dpp(v, 0x140, 0xf, 0xf, true));
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = up(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return up(b[0], b[1]);
}

// What the tokens of a workgroup become in LDS: codes [rows][P rounded up to 1024], zero behind the
// columns, and each row's scale and sum of codes.
struct Staged {
  uint8_t* codes;
  float* scale;
  int* sum;
  int pitch;
};

// A row by the T threads t = 0 .. T - 1 of a wavefront or (T = kRowsThreads) of the workgroup.
template <int QT, bool VEC, int T>
__device__ __forceinline__ void stage_row(const I8Product& p, int64_t row, int i, int t, const Staged& s,
                                          uint32_t* tops) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t top = 0;
  auto elements = [&](int c, float (&v)[8]) {
    numbers8(load8<QT, VEC>(p.raw, row * p.ldraw + c, p.cols - c), v);
    if (p.colf) {
      float f[8];
      numbers8(load8<QZ_F32, VEC>(p.colf, c, p.cols - c), f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= f[j];
    }
  };
  for (int c = 8 * t; c < p.cols; c += 8 * T) {
    float v[8];
    elements(c, v);
    top = top8(v, top);
  }
  top = lanes_top(top);
  if constexpr (T > 64) {
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
    __syncthreads();   // before the next row's
  }
  const RowScale sc = row_scale(top);
  int sum = 0;
  for (int c = 8 * t; c < s.pitch; c += 8 * T) {
    uint2 w = make_uint2(0, 0);
    if (c < p.cols) {
      float v[8], q[8];
      elements(c, v);
      w = codes8(v, sc, q);
      sum = add_codes(w.x, add_codes(w.y, sum));
    }
    *reinterpret_cast<uint2*>(s.codes + i * s.pitch + c) = w;
  }
  if (p.zeros) {
    sum = lanes_sum(sum);
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

// Rows first .. first + n - 1 of the tokens; all threads of the workgroup call it.
template <int QT, bool VEC>
__device__ __forceinline__ void stage_rows(const I8Product& p, int64_t first, int n, const Staged& s, uint32_t* tops) {
  const int tid = threadIdx.x;
  if constexpr (QT == kCodes) {
    for (int c = 16 * tid; c < n * s.pitch; c += 16 * kRowsThreads) {
      const int i = c / s.pitch, at = c % s.pitch;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (at < p.P) v = *reinterpret_cast<const uint4*>(p.X + (first + i) * p.P + at);
      *reinterpret_cast<uint4*>(s.codes + c) = v;
    }
    if (tid < n) {
      s.scale[tid] = p.sx[first + tid];
      s.sum[tid] = p.zeros ? p.xsum[first + tid] : 0;
    }
  } else if (n < 4) {   // a barrier or two a row; otherwise a wavefront a row
    for (int i = 0; i < n; ++i) stage_row<QT, VEC, kRowsThreads>(p, first + i, i, tid, s, tops);
  } else {
    for (int i = tid / 64; i < n; i += kRowsThreads / 64) stage_row<QT, VEC, 64>(p, first + i, i, tid & 63, s, tops);
  }
  __syncthreads();
}

// A wavefront has R rows of W (kGateUp: R / 2 gate rows and their up rows); N tokens for kPlain.
// Lane l has 16 bytes of every 1024 columns; blocks of U times 1024 columns of R rows are loaded one
// ahead, the first one before the tokens are staged.
template <Form FORM, int QT, bool VEC, int N, int R>
__global__ __launch_bounds__(kRowsThreads) void i8_rows_kernel(const I8Product p) {
  constexpr int U = R >= 8 ? 1 : 8 / R;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float xscale[QZ_ROUTE_MAX_TOP_K];
  __shared__ int xsums[QZ_ROUTE_MAX_TOP_K];
  __shared__ uint32_t tops[4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int kOut = FORM == kGateUp ? R / 2 : R;   // results of a wavefront (for each token)
  const int64_t r0 = (blockIdx.x * (int64_t)4 + wave) * kOut;
  const int pair = FORM == kGateUp ? blockIdx.y : 0;
  const int token = FORM == kDown ? blockIdx.y : 0;
  const int segments = FORM == kDown ? p.k : 1;
  const uint32_t P = static_cast<uint32_t>(p.P);
  const Staged s{smem, xscale, xsums, static_cast<int>(round_up(p.P, 1024))};

  auto expert_of = [&](int at) {   // -1: not here
    const int e = FORM == kPlain ? 0 : p.ids[at];
    return FORM == kPlain || (e >= 0 && e < p.E) ? e : -1;
  };
  if (FORM == kGateUp && expert_of(pair) < 0) return;   // nobody reads its hidden row
  const int64_t w_rows = (FORM == kGateUp ? 2 : 1) * p.d_o;
  auto row_of = [&](int i) {   // of the expert's
    const int64_t r = r0 + (FORM == kGateUp ? i % kOut : i);
    return (r < p.d_o ? r : p.d_o - 1) + (FORM == kGateUp && i >= kOut ? p.d_o : 0);
  };
  const int per = (s.pitch / 1024 + U - 1) / U, blocks = segments * per;
  auto load = [&](int b, i32x4 (&w)[R][U]) {
    int e = FORM == kPlain ? 0 : expert_of(FORM == kGateUp ? pair : token * p.k + b / per);
    if (e < 0) e = 0;
    const int8_t* base = p.W + e * w_rows * p.P;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int8_t* row = base + row_of(i) * p.P;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t c = static_cast<uint32_t>(b % per * U + u) * 1024 + 16 * lane;
        w[i][u] = *reinterpret_cast<const i32x4*>(row + (c < P ? c : 0));   // past the row: against zeros
      }
    }
  };
  int acc[R][N];
  float y = 0.f;   // kDown: of row `lane`
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int t = 0; t < N; ++t) acc[i][t] = 0;
  };
  // Lane l's sum of [i][t], l = i N + t.
  auto mine = [&] {
    int v = 0;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int t = 0; t < N; ++t) {
        const int total = lanes_sum(acc[i][t]);
        v = lane == i * N + t ? total : v;
      }
    return v;
  };
  auto use = [&](int b, const i32x4 (&w)[R][U]) {
    const int seg = b / per;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = (b % per * U + u) * 1024 + 16 * lane;
      if (U > 1 && c >= s.pitch) continue;
#pragma unroll
      for (int t = 0; t < N; ++t) {
        const i32x4 x = *reinterpret_cast<const i32x4*>(s.codes + (seg + t) * s.pitch + c);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][t] = __builtin_amdgcn_sdot4(w[i][u][j], x[j], acc[i][t], false);
      }
    }
    if constexpr (FORM == kDown) {
      if ((b + 1) % per == 0) {   // an expert's product, weighted
        const int e = expert_of(token * p.k + seg);
        const int a = mine();
        const int64_t r = e * w_rows + (r0 + lane < p.d_o ? r0 + lane : p.d_o - 1);
        if (lane < R && e >= 0)
          y += p.pair_weight[token * p.k + seg] *
               scaled(a, p.zeros ? p.zeros[r] - 128 : 0, xsums[seg], xscale[seg], p.sw[r], 0.f);
        clear();
      }
    }
  };
  i32x4 even[R][U], odd[R][U];
  load(0, even);
  stage_rows<QT, VEC>(p, FORM == kDown ? (int64_t)token * p.k : FORM == kGateUp ? pair / p.k : 0,
                      FORM == kDown ? p.k : N, s, tops);
  clear();
  for (int b = 0;;) {
    if (b + 1 < blocks) load(b + 1, odd);
    use(b, even);
    if (++b >= blocks) break;
    if (b + 1 < blocks) load(b + 1, even);
    use(b, odd);
    if (++b >= blocks) break;
  }
  if constexpr (FORM == kDown) {
    if (lane < R && r0 + lane < p.d_o)
      static_cast<uint16_t*>(p.Y)[token * p.ldy + r0 + lane] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(y));
  } else if constexpr (FORM == kGateUp) {
    const int a = mine();
    const int i = lane % kOut;
    const int64_t r = expert_of(pair) * w_rows + row_of(lane < R ? lane : 0);
    float v = 0.f;
    if (lane < R) v = scaled(a, p.zeros ? p.zeros[r] - 128 : 0, xsums[0], xscale[0], p.sw[r], 0.f);
    const float up = __shfl(v, lane + kOut);
    if (lane < kOut && r0 + i < p.d_o) static_cast<float*>(p.Y)[pair * p.ldy + r0 + i] = silu(v) * up;
  } else {
    const int a = mine();
    const int i = lane / N, t = lane % N;
    const int64_t r = r0 + i;
    if (lane < R * N && r < p.d_o) {
      const float v = scaled(a, p.zeros ? p.zeros[r] - 128 : 0, xsums[t], xscale[t], p.sw[r], p.bias ? p.bias[r] : 0.f);
      if (p.yt == QZ_BF16)
        static_cast<uint16_t*>(p.Y)[t * p.ldy + r] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
      else
        static_cast<float*>(p.Y)[t * p.ldy + r] = v;
    }
  }
}

template <Form FORM, int QT, bool VEC, int N, int R>
int launch_rows(const I8Product& p, int64_t y, hipStream_t s) {
  const int64_t rows = FORM == kDown ? p.k : N, lds = rows * round_up(p.P, 1024);
  constexpr int kOut = 4 * (FORM == kGateUp ? R / 2 : R);
  hipLaunchKernelGGL((i8_rows_kernel<FORM, QT, VEC, N, R>), dim3(static_cast<unsigned>(ceil_div(p.d_o, kOut)), static_cast<unsigned>(y)),
                     dim3(kRowsThreads), static_cast<size_t>(lds), s, p);
  return check_launch("i8_rows");
}

template <Form FORM, int QT, bool VEC>
int by_tokens(const I8Product& p, int64_t y, hipStream_t s) {
  if constexpr (FORM != kPlain) {
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

template <Form FORM>
int by_type(const I8Product& p, int64_t y, hipStream_t s) {
  if (!p.raw) {
    if constexpr (FORM != kGateUp) return by_tokens<FORM, kCodes, true>(p, y, s);
    return fail(QZ_EHIP, "i8_rows: no kernel");
  }
  const size_t size = p.rt == QZ_BF16 ? 2 : 4;
  auto on16 = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
  const bool vec = p.cols % 8 == 0 && p.ldraw * size % 16 == 0 && on16(p.raw) && on16(p.colf);
  if constexpr (FORM != kDown)
    if (p.rt == QZ_BF16)
      return vec ? by_tokens<FORM, QZ_BF16, true>(p, y, s) : by_tokens<FORM, QZ_BF16, false>(p, y, s);
  return vec ? by_tokens<FORM, QZ_F32, true>(p, y, s) : by_tokens<FORM, QZ_F32, false>(p, y, s);
}

}  // namespace

// LDS of a workgroup for the tokens' codes.
constexpr int64_t kRowsLds = 60 * 1024;

bool i8_rows_fits(int64_t rows, int64_t P) { return rows * round_up(P, 1024) <= kRowsLds; }

int launch_i8_rows(const I8Product& p, hipStream_t s) { return by_type<kPlain>(p, 1, s); }
int launch_i8_rows_gate_up(const I8Product& p, hipStream_t s) { return by_type<kGateUp>(p, p.n, s); }
int launch_i8_rows_down(const I8Product& p, int64_t tokens, hipStream_t s) { return by_type<kDown>(p, tokens, s); }

}  // namespace qz
