// C ABI of the microscaled 4-bit operators (declared and documented in include/qz.h):
// argument checks, workspace layout and launches.
#include <cstdint>
#include <string>

#include "mx4.h"

using namespace qz;

namespace {

// Launches index rows and tokens with 16-row grid rows and 32-bit grid dimensions.
constexpr int64_t kMaxRows = int64_t(1) << 24;
constexpr int64_t kMaxTokens = int64_t(1) << 20;
constexpr int64_t kMaxCols = int64_t(1) << 20;   // byte offsets of a 256-row tile fit 32 bits

bool float_type(int t) { return t == QZ_BF16 || t == QZ_F32; }
bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t type_size(int t) { return t == QZ_BF16 ? 2 : 4; }

int check_ws(const char* who, const void* ws, size_t have, size_t need) {
  if (have < need || (need > 0 && !ws))
    return fail(QZ_EWORKSPACE, std::string(who) + ": workspace too small");
  if (need > 0 && !aligned(ws, 256))
    return fail(QZ_EWORKSPACE, std::string(who) + ": workspace must be 256-byte aligned");
  return QZ_OK;
}

int check_codes(const char* who, const uint8_t* codes, const uint8_t* scales) {
  if (!codes || !scales) return fail(QZ_EINVAL, std::string(who) + ": null pointer");
  if (!aligned(codes, 16))
    return fail(QZ_EINVAL, std::string(who) + ": codes must be 16-byte aligned");
  return QZ_OK;
}

// Rows of X that the kernels read as they are: whole blocks on 16-byte boundaries.  Other
// rows are copied to the workspace first.
bool direct_x(const void* X, int64_t d_i, int64_t ldx) {
  return d_i % kMxBlock == 0 && ldx % 8 == 0 && ldx <= 2 * kMaxCols && aligned(X, 16);
}

// X's rows copied to whole blocks, and the sums of a split product.
struct ProductWs {
  uint16_t* xpad;
  float* partial;
  Mx4Choice choice;
  size_t bytes;
};
ProductWs product_ws(void* base, bool x4, bool pad, int64_t n, int64_t d_o, int64_t d_i) {
  Carver c(base);
  ProductWs w;
  w.xpad = c.take<uint16_t>(pad ? static_cast<size_t>(n) * mx_blocks(d_i) * kMxBlock : 0);
  w.choice = mx4_choose(x4, n, d_o, mx_blocks(d_i));
  const size_t splits = w.choice.splits;
  w.partial = c.take<float>(splits > 1 ? splits * n * d_o : 0);
  w.bytes = c.used;
  if (splits <= 1) w.partial = nullptr;
  return w;
}

bool product_sizes(int64_t n, int64_t d_o, int64_t d_i) {
  return n >= 0 && n <= kMaxTokens && d_o >= 0 && d_o <= kMaxRows && d_i >= 1 && d_i <= kMaxCols;
}

// What the kernels may assume of the output and of the factors.
void set_alignment(Mx4Product* p) {
  p->y_vec = p->ldy % 4 == 0 && aligned(p->Y, 4 * type_size(p->yt));
  p->factors_aligned = aligned(p->scales, 4) && aligned(p->xscales, 4);
}

struct MoeWs {
  double *logits, *top;
  int32_t *sel, *slot_expert, *slot_count, *slot_pairs;
  float* y_pairs;
  uint16_t *h_hi, *h_lo, *xpad;
  size_t bytes;
};
MoeWs moe_ws(void* base, int64_t n, int64_t d, int64_t f, const qz_moe* p) {
  Carver c(base);
  MoeWs w;
  const size_t pairs = static_cast<size_t>(n) * p->top_k;
  w.logits = c.take<double>(static_cast<size_t>(n) * p->n_experts);
  w.top = c.take<double>(pairs);
  w.sel = c.take<int32_t>(pairs);
  const size_t slots = static_cast<size_t>(moe_slots(n, p->n_experts, p->top_k));
  w.slot_expert = c.take<int32_t>(slots);
  w.slot_count = c.take<int32_t>(slots);
  w.slot_pairs = c.take<int32_t>(slots * n);
  w.y_pairs = c.take<float>(pairs * round_up(d, 4));
  w.h_hi = c.take<uint16_t>(pairs * mx_blocks(f) * kMxBlock);
  w.h_lo = c.take<uint16_t>(pairs * mx_blocks(f) * kMxBlock);
  w.xpad = c.take<uint16_t>(static_cast<size_t>(n) * mx_blocks(d) * kMxBlock);
  w.bytes = c.used;
  return w;
}

int check_moe(const qz_moe* p) {
  if (!p) return fail(QZ_EINVAL, "mx4_moe: params is null");
  if (p->struct_size < sizeof(qz_moe)) return fail(QZ_EINVAL, "mx4_moe: params.struct_size too small");
  if (p->n_experts < 1 || p->n_experts > QZ_MOE_MAX_EXPERTS)
    return fail(QZ_EINVAL, "mx4_moe: n_experts must be in 1..256");
  if (p->top_k < 1 || p->top_k > QZ_MOE_MAX_TOP_K || p->top_k > p->n_experts)
    return fail(QZ_EINVAL, "mx4_moe: top_k must be in 1..16 and at most n_experts");
  if (p->flags & ~QZ_MOE_RENORM) return fail(QZ_EINVAL, "mx4_moe: unknown flags");
  return QZ_OK;
}

bool moe_sizes(int64_t n, int64_t d, int64_t f) {
  return n >= 0 && n <= QZ_MOE_MAX_TOKENS && d >= 1 && d <= kMaxCols && f >= 1 && f <= (1 << 20);
}

}  // namespace

extern "C" {

int64_t qz_mx4_blocks(int64_t cols) { return cols < 1 ? -1 : mx_blocks(cols); }

int qz_mx4_quantize(const void* W, int32_t wt, int64_t rows, int64_t cols, int64_t ldw,
                    int32_t rule, const float* colw, uint8_t* codes, uint8_t* scales, void* values,
                    hipStream_t stream) {
  if (!float_type(wt)) return fail(QZ_EINVAL, "mx4_quantize: bad dtype");
  if (rows < 0 || cols < 1) return fail(QZ_EINVAL, "mx4_quantize: need rows >= 0 and cols >= 1");
  if (ldw < cols) return fail(QZ_EINVAL, "mx4_quantize: ldw must be at least cols");
  if (rule != QZ_MX4_FLOOR && rule != QZ_MX4_LEAST) return fail(QZ_EINVAL, "mx4_quantize: unknown rule");
  if (colw && rule != QZ_MX4_LEAST)
    return fail(QZ_EINVAL, "mx4_quantize: column weights need the rule QZ_MX4_LEAST");
  if (rows == 0) return QZ_OK;
  if (!W) return fail(QZ_EINVAL, "mx4_quantize: null pointer");
  QZ_TRY(check_codes("mx4_quantize", codes, scales));
  if (!aligned(W, type_size(wt)) || !aligned(values, type_size(wt)) || !aligned(colw, 4))
    return fail(QZ_EINVAL, "mx4_quantize: arrays must be aligned to their elements");
  set_error("");
  ScopedTimer tm(K_MX4_QUANTIZE, stream);
  return launch_mx4_quantize(W, wt, rows, cols, ldw, rule, colw, codes, scales, values, stream);
}

int qz_mx4_unpack(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                  int32_t* out, float* out_scales, uint8_t* zeros, hipStream_t stream) {
  if (rows < 0 || cols < 1) return fail(QZ_EINVAL, "mx4_unpack: need rows >= 0 and cols >= 1");
  if (rows == 0) return QZ_OK;
  QZ_TRY(check_codes("mx4_unpack", codes, scales));
  if (!out || !out_scales || !zeros) return fail(QZ_EINVAL, "mx4_unpack: null pointer");
  if (!aligned(out, 4) || !aligned(out_scales, 4))
    return fail(QZ_EINVAL, "mx4_unpack: arrays must be aligned to their elements");
  set_error("");
  ScopedTimer tm(K_MX4_QUANTIZE, stream);
  return launch_mx4_unpack(codes, scales, rows, cols, out, out_scales, zeros, stream);
}

static int check_product(const char* who, int64_t n, int64_t d_o, int64_t d_i,
                         const uint8_t* codes, const uint8_t* scales, const float* bias, void* Y,
                         int32_t yt, int64_t ldy) {
  const std::string w(who);
  if (!float_type(yt)) return fail(QZ_EINVAL, w + ": bad output dtype");
  if (!product_sizes(n, d_o, d_i))
    return fail(QZ_EINVAL, w + ": need 0 <= n <= 2^20, 0 <= d_o <= 2^24, 1 <= d_i <= 2^20");
  if (ldy < d_o) return fail(QZ_EINVAL, w + ": ldy must be at least d_o");
  if (n == 0 || d_o == 0) return QZ_OK;
  if (!Y) return fail(QZ_EINVAL, w + ": null pointer");
  QZ_TRY(check_codes(who, codes, scales));
  if (!aligned(Y, type_size(yt)) || !aligned(bias, 4))
    return fail(QZ_EINVAL, w + ": arrays must be aligned to their elements");
  return QZ_OK;
}

size_t qz_mx4_linear_workspace(const void* X, int64_t n, int64_t ldx, int64_t d_o, int64_t d_i) {
  if (!product_sizes(n, d_o, d_i)) return 0;
  return product_ws(nullptr, false, !X || !direct_x(X, d_i, ldx), n, d_o, d_i).bytes;
}

int qz_mx4_linear(const void* X, int32_t xt, int64_t n, int64_t ldx, const uint8_t* codes,
                  const uint8_t* scales, int64_t d_o, int64_t d_i, const float* bias, void* Y,
                  int32_t yt, int64_t ldy, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (xt != QZ_BF16) return fail(QZ_EINVAL, "mx4_linear: X must be bf16");
  QZ_TRY(check_product("mx4_linear", n, d_o, d_i, codes, scales, bias, Y, yt, ldy));
  if (ldx < d_i) return fail(QZ_EINVAL, "mx4_linear: ldx must be at least d_i");
  if (n == 0 || d_o == 0) return QZ_OK;
  if (!X) return fail(QZ_EINVAL, "mx4_linear: null pointer");
  if (!aligned(X, 2)) return fail(QZ_EINVAL, "mx4_linear: arrays must be aligned to their elements");
  const bool pad = !direct_x(X, d_i, ldx);
  const ProductWs w = product_ws(ws, false, pad, n, d_o, d_i);
  QZ_TRY(check_ws("mx4_linear", ws, ws_bytes, w.bytes));
  set_error("");
  ScopedTimer tm(K_MX4_PRODUCT, stream);
  Mx4Product p{};
  p.n = n;
  p.d_o = d_o;
  p.G = mx_blocks(d_i);
  p.X = static_cast<const uint16_t*>(X);
  p.ldx = ldx;
  p.choice = w.choice;
  p.partial = w.partial;
  if (pad) {
    p.ldx = p.G * kMxBlock;
    p.X = w.xpad;
    QZ_TRY(launch_mx4_pad(static_cast<const uint16_t*>(X), n, d_i, ldx, w.xpad, p.ldx, stream));
  }
  p.codes = codes;
  p.scales = scales;
  p.bias = bias;
  p.Y = Y;
  p.yt = yt;
  p.ldy = ldy;
  set_alignment(&p);
  return launch_mx4_product(p, stream);
}

size_t qz_mx4_matmul_workspace(int64_t n, int64_t d_o, int64_t d_i) {
  if (!product_sizes(n, d_o, d_i)) return 0;
  return product_ws(nullptr, true, false, n, d_o, d_i).bytes;
}

int qz_mx4_matmul(const uint8_t* xcodes, const uint8_t* xscales, int64_t n, const uint8_t* codes,
                  const uint8_t* scales, int64_t d_o, int64_t d_i, const float* bias, void* Y,
                  int32_t yt, int64_t ldy, void* ws, size_t ws_bytes, hipStream_t stream) {
  QZ_TRY(check_product("mx4_matmul", n, d_o, d_i, codes, scales, bias, Y, yt, ldy));
  if (n == 0 || d_o == 0) return QZ_OK;
  QZ_TRY(check_codes("mx4_matmul", xcodes, xscales));
  const ProductWs w = product_ws(ws, true, false, n, d_o, d_i);
  QZ_TRY(check_ws("mx4_matmul", ws, ws_bytes, w.bytes));
  set_error("");
  ScopedTimer tm(K_MX4_PRODUCT, stream);
  Mx4Product p{};
  p.n = n;
  p.d_o = d_o;
  p.G = mx_blocks(d_i);
  p.xcodes = xcodes;
  p.xscales = xscales;
  p.choice = w.choice;
  p.partial = w.partial;
  p.codes = codes;
  p.scales = scales;
  p.bias = bias;
  p.Y = Y;
  p.yt = yt;
  p.ldy = ldy;
  set_alignment(&p);
  return launch_mx4_product(p, stream);
}

size_t qz_mx4_moe_workspace(int64_t n, int64_t d, int64_t f, const qz_moe* params) {
  if (!moe_sizes(n, d, f) || check_moe(params) != QZ_OK) return 0;
  return moe_ws(nullptr, n, d, f, params).bytes;
}

int qz_mx4_moe(const void* X, int32_t xt, int64_t n, int64_t ldx, int64_t d, int64_t f,
               const qz_moe* params, const void* router, int32_t rt, const uint8_t* gu_codes,
               const uint8_t* gu_scales, const uint8_t* dn_codes, const uint8_t* dn_scales,
               void* Y, int32_t* ids, float* weights, void* ws, size_t ws_bytes,
               hipStream_t stream) {
  if (xt != QZ_BF16) return fail(QZ_EINVAL, "mx4_moe: X must be bf16");
  if (!float_type(rt)) return fail(QZ_EINVAL, "mx4_moe: bad router dtype");
  QZ_TRY(check_moe(params));
  if (!moe_sizes(n, d, f))
    return fail(QZ_EINVAL, "mx4_moe: need 0 <= n <= 256, 1 <= d <= 2^20, 1 <= f <= 2^20");
  if (ldx < d) return fail(QZ_EINVAL, "mx4_moe: ldx must be at least d");
  if (n == 0) return QZ_OK;
  if (!X || !router || !Y) return fail(QZ_EINVAL, "mx4_moe: null pointer");
  QZ_TRY(check_codes("mx4_moe", gu_codes, gu_scales));
  QZ_TRY(check_codes("mx4_moe", dn_codes, dn_scales));
  if (!aligned(X, 2) || !aligned(Y, 2) || !aligned(router, type_size(rt)) || !aligned(ids, 4) ||
      !aligned(weights, 4))
    return fail(QZ_EINVAL, "mx4_moe: arrays must be aligned to their elements");
  const MoeWs w = moe_ws(ws, n, d, f, params);
  QZ_TRY(check_ws("mx4_moe", ws, ws_bytes, w.bytes));
  set_error("");
  ScopedTimer tm(K_MX4_MOE, stream);
  MoeArgs a{};
  a.n = n;
  a.d = d;
  a.f = f;
  a.Gd = mx_blocks(d);
  a.Gf = mx_blocks(f);
  a.E = params->n_experts;
  a.k = params->top_k;
  a.renorm = (params->flags & QZ_MOE_RENORM) != 0;
  a.X = static_cast<const uint16_t*>(X);
  a.ldx = ldx;
  if (!direct_x(X, d, ldx)) {
    a.ldx = a.Gd * kMxBlock;
    a.X = w.xpad;
    QZ_TRY(launch_mx4_pad(static_cast<const uint16_t*>(X), n, d, ldx, w.xpad, a.ldx, stream));
  }
  a.router = router;
  a.gu_codes = gu_codes;
  a.gu_scales = gu_scales;
  a.dn_codes = dn_codes;
  a.dn_scales = dn_scales;
  a.Y = static_cast<uint16_t*>(Y);
  a.ids = ids;
  a.weights = weights;
  a.logits = w.logits;
  a.sel = w.sel;
  a.top = w.top;
  a.h_hi = w.h_hi;
  a.h_lo = w.h_lo;
  a.ldh = a.Gf * kMxBlock;
  a.slot_expert = w.slot_expert;
  a.slot_count = w.slot_count;
  a.slot_pairs = w.slot_pairs;
  a.y_pairs = w.y_pairs;
  a.ldy = round_up(d, 4);
  return launch_moe(a, rt, stream);
}

}  // extern "C"
