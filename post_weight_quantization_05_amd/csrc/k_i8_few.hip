// Products of 8-bit integer rows with few tokens: workgroups of 16 RT rows of W by 16 NT tokens, whose
// wavefronts share the contraction.
//
// With few tokens W is read once and little is computed on it, so what counts is how many bytes are on
// their way.  There are too few tiles to fill the chip with a wavefront each, so the four wavefronts of a
// workgroup split the contraction and add their sums in LDS at the end; each has a ring of stages of its
// own, of 128 columns (whole lines), and waits for its own copies alone, without a barrier.  13 tokens
// 12288 -> 4096: 49 MB of W in 10.6 us (4.9 TB/s with the launch), 256 workgroups, 20 KB of copies a
// wavefront on their way; 64 tokens 4096 -> 4096 6.3 us, against 9.2 by tiles.
#include <type_traits>

#include "i8_gemm.h"
#include "i8_plan.h"
#include "lds_copy.h"

namespace qz {

namespace {

// Until at most N copies of this wavefront are in flight.
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
  asm volatile("" ::: "memory");
}

template <Form FORM, class T>
__global__ __launch_bounds__(64 * T::kWaves) void i8_few_kernel(const I8Product p) {
  constexpr int RT = T::RT, NT = T::NT, D = T::kDepth;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  lds_u8* const lds = (lds_u8*)smem + wave * D * T::kStage;
  int expert = 0, slot0 = 0, slot_end = 0;
  if constexpr (FORM != kPlain) {
    const Tiles tiles(p, 16 * NT);
    if (static_cast<int>(blockIdx.y) >= tiles.total) return;
    tiles.find(blockIdx.y, 16 * NT, &expert, &slot0, &slot_end);
  }
  const int64_t t0 = FORM == kPlain ? blockIdx.y * (int64_t)(16 * NT) : slot0;
  const int64_t t_end = FORM == kPlain ? p.n : slot_end;
  constexpr int kRows = FORM == kGateUp ? 8 * RT : 16 * RT;   // output rows
  const int64_t r0 = blockIdx.x * (int64_t)kRows;
  const int last_r = static_cast<int>(p.d_o - 1 - r0 < kRows ? p.d_o - 1 - r0 : kRows);
  const int last_t = static_cast<int>(t_end - 1 - t0 < 16 * NT ? t_end - 1 - t0 : 16 * NT);
  const int64_t w_row0 = static_cast<int64_t>(expert) * (FORM == kGateUp ? 2 : 1) * p.d_o;

  const int all = static_cast<int>(p.P / 128), mine = (all + T::kWaves - 1) / T::kWaves;
  const int first = wave * mine;
  const int nst = all - first < mine ? all - first : mine;   // <= 0: none
  const uint32_t pitch = static_cast<uint32_t>(p.P);
  uint32_t from_w[2 * RT], from_x[2 * NT];
#pragma unroll
  for (int i = 0; i < 2 * RT; ++i) {
    const int r = 8 * i + lane / 8, chunk = (lane % 8) ^ swz<128>(r);
    const int o = FORM == kGateUp ? r % kRows : r;
    const uint32_t row = (o < last_r ? o : last_r) + (FORM == kGateUp && r >= kRows ? static_cast<uint32_t>(p.d_o) : 0u);
    from_w[i] = row * pitch + 16 * chunk;
  }
#pragma unroll
  for (int i = 0; i < 2 * NT; ++i) {
    const int r = 8 * i + lane / 8, chunk = (lane % 8) ^ swz<128>(r);
    uint32_t row = r < last_t ? r : last_t;
    if constexpr (FORM == kGateUp) row = static_cast<uint32_t>(p.order[t0 + row]) / static_cast<uint32_t>(p.k);
    from_x[i] = row * pitch + 16 * chunk;
  }
  const uint8_t* const wbase = reinterpret_cast<const uint8_t*>(p.W) + (w_row0 + r0) * p.P + static_cast<int64_t>(first) * 128;
  const uint8_t* const xbase = reinterpret_cast<const uint8_t*>(p.X) + (FORM == kGateUp ? 0 : t0 * p.P) + static_cast<int64_t>(first) * 128;
  auto issue = [&](int st, int slot) {
    lds_u8* const at = lds + slot * T::kStage;
#pragma unroll
    for (int i = 0; i < 2 * RT; ++i) copy_lds<16>(at + i * 1024, wbase + static_cast<int64_t>(st) * 128, from_w[i]);
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) copy_lds<16>(at + (2 * RT + i) * 1024, xbase + static_cast<int64_t>(st) * 128, from_x[i]);
  };
  i32x4 acc[RT][NT];
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int b = 0; b < NT; ++b) acc[a][b] = i32x4{0, 0, 0, 0};
  const int m = lane & 15, q = lane >> 4;
  auto rd16 = [](lds_u8* at) { return *(__attribute__((address_space(3))) i32x4*)at; };
  auto products = [&](int slot) {
    lds_u8* const at = lds + slot * T::kStage + m * 128;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int c = 16 * ((4 * s + q) ^ swz<128>(m));
      i32x4 w[RT], x[NT];
#pragma unroll
      for (int a = 0; a < RT; ++a) w[a] = rd16(at + a * 2048 + c);
#pragma unroll
      for (int b = 0; b < NT; ++b) x[b] = rd16(at + (RT + b) * 2048 + c);
#pragma unroll
      for (int a = 0; a < RT; ++a)
#pragma unroll
        for (int b = 0; b < NT; ++b) acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[a], x[b], acc[a][b], 0, 0, 0);
    }
  };
#pragma unroll
  for (int i = 0; i < D; ++i)
    if (i < nst) issue(i, i);
  // The products of stage st have read their operands out of LDS before its place is filled again.
  int slot = 0, st = 0;
  for (; st + D < nst; ++st) {
    wait_copies<(D - 1) * T::kCopies>();
    products(slot);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    issue(st + D, slot);
    slot = slot + 1 < D ? slot + 1 : 0;
  }
  wait_copies<0>();
  for (; st < nst; ++st) {
    products(slot);
    slot = slot + 1 < D ? slot + 1 : 0;
  }

  // The wavefronts' sums, through LDS: of tile (a, b), lane l has token l % 16, rows 4 (l / 16) + i.
  __syncthreads();
  lds_u8* const part = (lds_u8*)smem;
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int b = 0; b < NT; ++b)
      *(__attribute__((address_space(3))) i32x4*)(part + ((wave * RT + a) * NT + b) * 1024 + 16 * lane) = acc[a][b];
  __syncthreads();
  auto total = [&](int a, int b) {
    i32x4 v = {0, 0, 0, 0};
    for (int w = 0; w < T::kWaves; ++w) v += rd16(part + ((w * RT + a) * NT + b) * 1024 + 16 * lane);
    return v;
  };
  constexpr int kTiles = kRows / 16 * NT;
  const bool vec = p.ldy % 4 == 0 && reinterpret_cast<uintptr_t>(p.Y) % 16 == 0;
  for (int i = wave; i < kTiles; i += T::kWaves) {
    const int a = i / NT, b = i % NT;
    const int64_t slot_at = t0 + 16 * b + m, r = r0 + 16 * a + 4 * q;
    const i32x4 sum = total(a, b);
    i32x4 up = {0, 0, 0, 0};
    if constexpr (FORM == kGateUp) up = total(a + RT / 2, b);
    if (slot_at >= t_end || r >= p.d_o) continue;
    const int64_t pair = FORM == kPlain ? slot_at : p.order[slot_at];
    const int64_t xr = FORM == kGateUp ? pair / p.k : slot_at;
    const float sx = p.sx[xr];
    const int xsum = p.zeros ? p.xsum[xr] : 0;
    f32x4 v, u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = w_row0 + (r + j < p.d_o ? r + j : p.d_o - 1);
      v[j] = scaled(sum[j], p.zeros ? p.zeros[c] - 128 : 0, xsum, sx, p.sw[c], FORM == kPlain && p.bias ? p.bias[c] : 0.f);
      if constexpr (FORM == kGateUp) {
        const int64_t cu = c + p.d_o;
        u[j] = scaled(up[j], p.zeros ? p.zeros[cu] - 128 : 0, xsum, sx, p.sw[cu], 0.f);
      }
    }
    if constexpr (FORM == kGateUp) v = silu(v) * u;
    if constexpr (FORM == kDown) v *= p.pair_weight[pair];
    const int64_t at = (FORM == kDown ? pair : slot_at) * p.ldy + r;
    const bool whole = vec && r + 4 <= p.d_o;
    if (FORM == kPlain && p.yt == QZ_BF16) {
      uint16_t* o = static_cast<uint16_t*>(p.Y) + at;
      const uint2 w = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
      if (whole) {
        *reinterpret_cast<uint2*>(o) = w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (r + j < p.d_o) o[j] = static_cast<uint16_t>((j < 2 ? w.x : w.y) >> (16 * (j % 2)));
      }
    } else {
      float* o = static_cast<float*>(p.Y) + at;
      if (whole) {
        *reinterpret_cast<f32x4*>(o) = v;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (r + j < p.d_o) o[j] = v[j];
      }
    }
  }
}

}  // namespace

template <Form FORM, class T>
static int launch_few(const I8Product& p, hipStream_t s) {
  const auto kernel = i8_few_kernel<FORM, T>;
  static LdsAllowance allowed;
  QZ_TRY(allowed.ask(reinterpret_cast<const void*>(kernel), T::kLds));
  const int64_t tiles = FORM == kPlain ? ceil_div(p.n, 16 * T::NT) : most_tiles(p, 16 * T::NT);
  if (tiles > 65535) return fail(QZ_EINVAL, "i8_few: too many tokens");
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(ceil_div(p.d_o, FORM == kGateUp ? 8 * T::RT : 16 * T::RT)), static_cast<unsigned>(tiles)),
                     dim3(64 * T::kWaves), T::kLds, s, p);
  return check_launch("i8_few");
}

template <Form FORM>
static int by_kind(I8Kind kind, const I8Product& p, hipStream_t s) {
  switch (kind) {
    case I8Kind::kFew11: if constexpr (FORM != kGateUp) return launch_few<FORM, Few11>(p, s); break;
    case I8Kind::kFew21: return launch_few<FORM, Few21>(p, s);
    case I8Kind::kFew22: return launch_few<FORM, Few22>(p, s);
    case I8Kind::kFew24: return launch_few<FORM, Few24>(p, s);
    default: break;
  }
  return fail(QZ_EHIP, "i8_few: no kernel");
}

int launch_i8_few(I8Kind kind, int form, const I8Product& p, hipStream_t s) {
  return form == kPlain ? by_kind<kPlain>(kind, p, s) : form == kGateUp ? by_kind<kGateUp>(kind, p, s) : by_kind<kDown>(kind, p, s);
}

}  // namespace qz
