// C ABI of the 8-bit integer operators and the router (declared and documented in include/qz.h):
// argument checks, workspace layout and launches.
#include <cmath>
#include <cstdint>
#include <string>

#include "i8_plan.h"
#include "qz_internal.h"

using namespace qz;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 24;     // of W
constexpr int64_t kMaxTokens = int64_t(1) << 20;
// The codes of an expert layer's tokens, and of an expert's gate rows: 32-bit offsets reach the up rows.
constexpr int64_t kMaxLayerBytes = int64_t(1) << 31;

bool float_type(int t) { return t == QZ_BF16 || t == QZ_F32; }
bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t type_size(int t) { return t == QZ_BF16 ? 2 : 4; }
bool cols_ok(int64_t cols) { return cols >= 1 && cols <= QZ_I8_MAX_COLS; }

int check_ws(const char* who, const void* ws, size_t have, size_t need) {
  if (have < need || (need > 0 && !ws))
    return fail(QZ_EWORKSPACE, std::string(who) + ": workspace too small");
  if (need > 0 && !aligned(ws, 256))
    return fail(QZ_EWORKSPACE, std::string(who) + ": workspace must be 256-byte aligned");
  return QZ_OK;
}

int check_codes(const char* who, const int8_t* codes, const float* scales) {
  if (!codes || !scales) return fail(QZ_EINVAL, std::string(who) + ": null pointer");
  if (!aligned(codes, 16)) return fail(QZ_EINVAL, std::string(who) + ": codes must be 16-byte aligned");
  if (!aligned(scales, 4))
    return fail(QZ_EINVAL, std::string(who) + ": arrays must be aligned to their elements");
  return QZ_OK;
}

bool product_sizes(int64_t n, int64_t d_o, int64_t d_i) {
  return n >= 0 && n <= kMaxTokens && d_o >= 0 && d_o <= kMaxRows && cols_ok(d_i);
}

int check_product(const char* who, int64_t n, int64_t d_o, int64_t d_i, const int8_t* codes,
                  const float* scales, const float* bias, void* Y, int32_t yt, int64_t ldy) {
  const std::string w(who);
  if (!float_type(yt)) return fail(QZ_EINVAL, w + ": bad output dtype");
  if (!product_sizes(n, d_o, d_i))
    return fail(QZ_EINVAL, w + ": need 0 <= n <= 2^20, 0 <= d_o <= 2^24, 1 <= d_i <= 65536");
  if (ldy < d_o) return fail(QZ_EINVAL, w + ": ldy must be at least d_o");
  if (n == 0 || d_o == 0) return QZ_OK;
  if (!Y) return fail(QZ_EINVAL, w + ": null pointer");
  QZ_TRY(check_codes(who, codes, scales));
  if (!aligned(Y, type_size(yt)) || !aligned(bias, 4))
    return fail(QZ_EINVAL, w + ": arrays must be aligned to their elements");
  return QZ_OK;
}

// X quantized.
struct LinearWs {
  int8_t* codes;
  float* scales;
  int32_t* sums;
  size_t bytes;
};
LinearWs linear_ws(void* base, int64_t n, int64_t d_i) {
  Carver c(base);
  LinearWs w{};
  if (i8_by_rows(n, i8_pitch(d_i))) return w;
  w.codes = c.take<int8_t>(static_cast<size_t>(n) * i8_pitch(d_i));
  w.scales = c.take<float>(n);
  w.sums = c.take<int32_t>(n);
  w.bytes = c.used;
  return w;
}

struct MoeWs {
  int8_t *xcodes, *hcodes;
  float *xscales, *hscales, *h, *y;
  int32_t *xsums, *hsums, *offsets, *order;
  size_t bytes;
};
MoeWs moe_ws(void* base, int64_t n, int64_t d, int64_t f, int E, int k) {
  Carver c(base);
  MoeWs w{};
  const size_t pairs = static_cast<size_t>(n) * k;
  w.h = c.take<float>(pairs * round_up(f, 4));
  if (i8_moe_by_rows(n, d, f, E, k)) {
    w.bytes = c.used;
    return w;
  }
  w.xcodes = c.take<int8_t>(static_cast<size_t>(n) * i8_pitch(d));
  w.xscales = c.take<float>(n);
  w.xsums = c.take<int32_t>(n);
  w.offsets = c.take<int32_t>(E + 1);
  w.order = c.take<int32_t>(pairs);
  w.hcodes = c.take<int8_t>(pairs * i8_pitch(f));
  w.hscales = c.take<float>(pairs);
  w.hsums = c.take<int32_t>(pairs);
  w.y = c.take<float>(pairs * round_up(d, 4));
  w.bytes = c.used;
  return w;
}

int check_moe(int64_t n, int64_t d, int64_t f, int32_t E, int32_t k) {
  if (E < 1 || E > QZ_ROUTE_MAX_EXPERTS) return fail(QZ_EINVAL, "i8_moe: n_experts must be in 1..512");
  if (k < 1 || k > QZ_ROUTE_MAX_TOP_K) return fail(QZ_EINVAL, "i8_moe: top_k must be in 1..16");
  if (n < 0 || n > kMaxTokens || !cols_ok(d) || !cols_ok(f))
    return fail(QZ_EINVAL, "i8_moe: need 0 <= n <= 2^20, 1 <= d <= 65536, 1 <= f <= 65536");
  if (n * i8_pitch(d) >= kMaxLayerBytes)
    return fail(QZ_EINVAL, "i8_moe: n pitch(d) must be below 2^31 (more tokens: in parts)");
  if (f * i8_pitch(d) >= kMaxLayerBytes) return fail(QZ_EINVAL, "i8_moe: f pitch(d) must be below 2^31");
  return QZ_OK;
}

}  // namespace

extern "C" {

int64_t qz_i8_pitch(int64_t cols) { return cols_ok(cols) ? i8_pitch(cols) : -1; }

int qz_i8_quantize(const void* X, int32_t xt, int64_t rows, int64_t cols, int64_t ldx,
                   const float* colf, int8_t* codes, float* scales, int32_t* sums, void* values,
                   hipStream_t stream) {
  if (!float_type(xt)) return fail(QZ_EINVAL, "i8_quantize: bad dtype");
  if (rows < 0 || rows > kMaxRows || !cols_ok(cols))
    return fail(QZ_EINVAL, "i8_quantize: need 0 <= rows <= 2^24 and 1 <= cols <= 65536");
  if (ldx < cols) return fail(QZ_EINVAL, "i8_quantize: ldx must be at least cols");
  if (rows == 0) return QZ_OK;
  if (!X) return fail(QZ_EINVAL, "i8_quantize: null pointer");
  QZ_TRY(check_codes("i8_quantize", codes, scales));
  if (!aligned(X, type_size(xt)) || !aligned(values, type_size(xt)) || !aligned(colf, 4) || !aligned(sums, 4))
    return fail(QZ_EINVAL, "i8_quantize: arrays must be aligned to their elements");
  set_error("");
  ScopedTimer tm(K_I8_QUANTIZE, stream);
  return launch_i8_quantize(X, xt, rows, cols, ldx, colf, codes, scales, sums, values, stream);
}

int qz_i8_pack(const uint8_t* codes, int64_t rows, int64_t cols, int8_t* out, hipStream_t stream) {
  if (rows < 0 || rows > kMaxRows || !cols_ok(cols))
    return fail(QZ_EINVAL, "i8_pack: need 0 <= rows <= 2^24 and 1 <= cols <= 65536");
  if (rows == 0) return QZ_OK;
  if (!codes || !out) return fail(QZ_EINVAL, "i8_pack: null pointer");
  if (!aligned(out, 16)) return fail(QZ_EINVAL, "i8_pack: codes must be 16-byte aligned");
  set_error("");
  ScopedTimer tm(K_I8_QUANTIZE, stream);
  return launch_i8_pack(codes, rows, cols, out, stream);
}

int qz_i8_unpack(const int8_t* codes, int64_t rows, int64_t cols, uint8_t* out, hipStream_t stream) {
  if (rows < 0 || rows > kMaxRows || !cols_ok(cols))
    return fail(QZ_EINVAL, "i8_unpack: need 0 <= rows <= 2^24 and 1 <= cols <= 65536");
  if (rows == 0) return QZ_OK;
  if (!codes || !out) return fail(QZ_EINVAL, "i8_unpack: null pointer");
  if (!aligned(codes, 16)) return fail(QZ_EINVAL, "i8_unpack: codes must be 16-byte aligned");
  set_error("");
  ScopedTimer tm(K_I8_QUANTIZE, stream);
  return launch_i8_unpack(codes, rows, cols, out, stream);
}

size_t qz_i8_matmul_workspace(int64_t, int64_t, int64_t) { return 0; }   // no kernel of the products has one

int qz_i8_matmul(const int8_t* xcodes, const float* xscales, const int32_t* xsums, int64_t n,
                 const int8_t* codes, const float* scales, const uint8_t* zeros, int64_t d_o,
                 int64_t d_i, const float* bias, void* Y, int32_t yt, int64_t ldy, void*, size_t,
                 hipStream_t stream) {
  QZ_TRY(check_product("i8_matmul", n, d_o, d_i, codes, scales, bias, Y, yt, ldy));
  if (n == 0 || d_o == 0) return QZ_OK;
  QZ_TRY(check_codes("i8_matmul", xcodes, xscales));
  if (zeros && !xsums) return fail(QZ_EINVAL, "i8_matmul: zeros need the row sums of X");
  if (!aligned(xsums, 4)) return fail(QZ_EINVAL, "i8_matmul: arrays must be aligned to their elements");
  set_error("");
  ScopedTimer tm(K_I8_PRODUCT, stream);
  I8Product p{};
  p.n = n;
  p.d_o = d_o;
  p.P = i8_pitch(d_i);
  p.X = xcodes;
  p.sx = xscales;
  p.xsum = xsums;
  p.W = codes;
  p.sw = scales;
  p.zeros = zeros;
  p.bias = bias;
  p.Y = Y;
  p.yt = yt;
  p.ldy = ldy;
  return i8_by_rows(n, p.P) ? launch_i8_rows(p, stream) : launch_i8_product(p, stream);
}

size_t qz_i8_linear_workspace(int64_t n, int64_t d_o, int64_t d_i) {
  return product_sizes(n, d_o, d_i) ? linear_ws(nullptr, n, d_i).bytes : 0;
}

int qz_i8_linear(const void* X, int32_t xt, int64_t n, int64_t ldx, const float* colf,
                 const int8_t* codes, const float* scales, const uint8_t* zeros, int64_t d_o,
                 int64_t d_i, const float* bias, void* Y, int32_t yt, int64_t ldy, void* ws,
                 size_t ws_bytes, hipStream_t stream) {
  if (!float_type(xt)) return fail(QZ_EINVAL, "i8_linear: bad dtype");
  QZ_TRY(check_product("i8_linear", n, d_o, d_i, codes, scales, bias, Y, yt, ldy));
  if (ldx < d_i) return fail(QZ_EINVAL, "i8_linear: ldx must be at least d_i");
  if (n == 0 || d_o == 0) return QZ_OK;
  if (!X) return fail(QZ_EINVAL, "i8_linear: null pointer");
  if (!aligned(X, type_size(xt)) || !aligned(colf, 4))
    return fail(QZ_EINVAL, "i8_linear: arrays must be aligned to their elements");
  const LinearWs w = linear_ws(ws, n, d_i);
  QZ_TRY(check_ws("i8_linear", ws, ws_bytes, w.bytes));
  set_error("");
  ScopedTimer tm(K_I8_PRODUCT, stream);
  I8Product p{};
  p.n = n;
  p.d_o = d_o;
  p.P = i8_pitch(d_i);
  p.X = w.codes;
  p.sx = w.scales;
  p.xsum = w.sums;
  p.W = codes;
  p.sw = scales;
  p.zeros = zeros;
  p.bias = bias;
  p.Y = Y;
  p.yt = yt;
  p.ldy = ldy;
  if (i8_by_rows(n, p.P)) {
    p.raw = X;
    p.rt = xt;
    p.ldraw = ldx;
    p.cols = d_i;
    p.colf = colf;
    return launch_i8_rows(p, stream);
  }
  QZ_TRY(launch_i8_quantize(X, xt, n, d_i, ldx, colf, w.codes, w.scales, zeros ? w.sums : nullptr, nullptr, stream));
  return launch_i8_product(p, stream);
}

int qz_route(const void* logits, int32_t lt, int64_t n, int64_t ldl, const qz_router* params,
             const float* bias, int32_t* ids, float* weights, hipStream_t stream) {
  if (!float_type(lt)) return fail(QZ_EINVAL, "route: bad dtype");
  if (!params) return fail(QZ_EINVAL, "route: params is null");
  if (params->struct_size < sizeof(qz_router)) return fail(QZ_EINVAL, "route: params.struct_size too small");
  const qz_router p = *params;
  if (p.n_experts < 1 || p.n_experts > QZ_ROUTE_MAX_EXPERTS)
    return fail(QZ_EINVAL, "route: n_experts must be in 1..512");
  if (p.n_groups < 1 || p.n_groups > QZ_ROUTE_MAX_GROUPS || p.n_experts % p.n_groups)
    return fail(QZ_EINVAL, "route: n_groups must be in 1..64 and divide n_experts");
  if (p.top_groups < 1 || p.top_groups > p.n_groups)
    return fail(QZ_EINVAL, "route: top_groups must be in 1..n_groups");
  if (p.group_best < 1 || p.group_best > 2) return fail(QZ_EINVAL, "route: group_best must be 1 or 2");
  if (p.top_k < 1 || p.top_k > QZ_ROUTE_MAX_TOP_K || p.top_k > p.top_groups * (p.n_experts / p.n_groups))
    return fail(QZ_EINVAL, "route: top_k must be in 1..16 and at most the experts of top_groups groups");
  if (p.flags & ~(QZ_ROUTE_SIGMOID | QZ_ROUTE_RENORM)) return fail(QZ_EINVAL, "route: unknown flags");
  if (!std::isfinite(p.scale)) return fail(QZ_EINVAL, "route: scale must be finite");
  if (n < 0 || n > kMaxRows) return fail(QZ_EINVAL, "route: need 0 <= n <= 2^24");
  if (ldl < p.n_experts) return fail(QZ_EINVAL, "route: ldl must be at least n_experts");
  if (n == 0) return QZ_OK;
  if (!logits || !ids || !weights) return fail(QZ_EINVAL, "route: null pointer");
  if (!aligned(logits, type_size(lt)) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
    return fail(QZ_EINVAL, "route: arrays must be aligned to their elements");
  set_error("");
  ScopedTimer tm(K_ROUTE, stream);
  return launch_route(logits, lt, n, ldl, p, bias, ids, weights, stream);
}

size_t qz_i8_moe_workspace(int64_t n, int64_t d, int64_t f, int32_t n_experts, int32_t top_k) {
  return check_moe(n, d, f, n_experts, top_k) == QZ_OK ? moe_ws(nullptr, n, d, f, n_experts, top_k).bytes : 0;
}

int qz_i8_moe(const void* X, int32_t xt, int64_t n, int64_t ldx, int64_t d, int64_t f,
              int32_t n_experts, int32_t top_k, const int32_t* ids, const float* weights,
              const int8_t* gu_codes, const float* gu_scales, const uint8_t* gu_zeros,
              const int8_t* dn_codes, const float* dn_scales, const uint8_t* dn_zeros, void* Y,
              void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!float_type(xt)) return fail(QZ_EINVAL, "i8_moe: bad dtype");
  QZ_TRY(check_moe(n, d, f, n_experts, top_k));
  if (ldx < d) return fail(QZ_EINVAL, "i8_moe: ldx must be at least d");
  if (n == 0) return QZ_OK;
  if (!X || !ids || !weights || !Y) return fail(QZ_EINVAL, "i8_moe: null pointer");
  QZ_TRY(check_codes("i8_moe", gu_codes, gu_scales));
  QZ_TRY(check_codes("i8_moe", dn_codes, dn_scales));
  if (!aligned(X, type_size(xt)) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(Y, 2))
    return fail(QZ_EINVAL, "i8_moe: arrays must be aligned to their elements");
  const MoeWs w = moe_ws(ws, n, d, f, n_experts, top_k);
  QZ_TRY(check_ws("i8_moe", ws, ws_bytes, w.bytes));
  set_error("");
  ScopedTimer tm(K_I8_MOE, stream);
  const int64_t pairs = n * top_k;
  I8Product p{};
  p.n = pairs;
  p.offsets = w.offsets;
  p.order = w.order;
  p.pair_weight = weights;
  p.E = n_experts;
  p.k = top_k;
  p.d_o = f;
  p.P = i8_pitch(d);
  p.X = w.xcodes;
  p.sx = w.xscales;
  p.xsum = w.xsums;
  p.W = gu_codes;
  p.sw = gu_scales;
  p.zeros = gu_zeros;
  p.Y = w.h;
  p.yt = QZ_F32;
  p.ldy = round_up(f, 4);
  if (i8_moe_by_rows(n, d, f, n_experts, top_k)) {
    p.ids = ids;
    p.raw = X;
    p.rt = xt;
    p.ldraw = ldx;
    p.cols = d;
    QZ_TRY(launch_i8_rows_gate_up(p, stream));
    p.raw = w.h;
    p.rt = QZ_F32;
    p.ldraw = p.ldy;
    p.cols = f;
  } else {
    QZ_TRY(launch_i8_quantize_group(X, xt, n, d, ldx, w.xcodes, w.xscales, gu_zeros ? w.xsums : nullptr, ids, top_k,
                                    n_experts, w.offsets, w.order, stream));
    QZ_TRY(launch_i8_gate_up(p, stream));
    QZ_TRY(launch_i8_quantize(w.h, QZ_F32, pairs, f, p.ldy, nullptr, w.hcodes, w.hscales, dn_zeros ? w.hsums : nullptr, nullptr,
                              stream));
  }
  p.d_o = d;
  p.P = i8_pitch(f);
  p.X = w.hcodes;
  p.sx = w.hscales;
  p.xsum = w.hsums;
  p.W = dn_codes;
  p.sw = dn_scales;
  p.zeros = dn_zeros;
  if (i8_moe_by_rows(n, d, f, n_experts, top_k)) {
    p.Y = Y;
    p.ldy = d;
    return launch_i8_rows_down(p, n, stream);
  }
  p.Y = w.y;
  p.ldy = round_up(d, 4);
  QZ_TRY(launch_i8_down(p, stream));
  return launch_i8_sum(w.y, p.ldy, ids, n, d, top_k, n_experts, static_cast<uint16_t*>(Y), stream);
}

}  // extern "C"
