// Native calls of the 8-bit integer operators and the router from Python.
//
// A call on few rows keeps the GPU busy for 3 to 5 us, and the interpreter's part of it (a look at every
// tensor, the foreign call, the result's allocation) took as long again.  Each function here does that part
// for the ordinary call: it checks what the package's Python checks, allocates the results and calls the
// library.  For anything else (another GPU than the current one, a bad argument, an error status) it returns
// None, and the Python code makes the call, or says what is wrong with it.
//
// The library's functions come by address (init), so this module links nothing of it.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "qz.h"

namespace {

struct {
  decltype(&qz_i8_quantize) quantize;
  decltype(&qz_i8_matmul_workspace) matmul_workspace;
  decltype(&qz_i8_matmul) matmul;
  decltype(&qz_i8_linear_workspace) linear_workspace;
  decltype(&qz_i8_linear) linear;
  decltype(&qz_route) route;
  decltype(&qz_i8_moe_workspace) moe_workspace;
  decltype(&qz_i8_moe) moe;
} lib;

// Thrown for a call that is left to Python.
struct Leave {};
void need(bool ok) {
  if (!ok) throw Leave{};
}

const at::Tensor& tensor(PyObject* o) {
  need(THPVariable_Check(o));
  return THPVariable_Unpack(o);
}

// A tensor on GPU `index`, plainly strided.
const at::Tensor& on(PyObject* o, int64_t index, at::ScalarType type) {
  const at::Tensor& t = tensor(o);
  need(t.is_cuda() && t.get_device() == index && t.layout() == at::kStrided && t.scalar_type() == type);
  return t;
}

struct Matrix {
  const void* p;
  int64_t rows, cols, ld, index;
  int32_t type;
};
// Contiguous rows that do not overlap, bf16 or fp32, on the current GPU.
Matrix matrix(const at::Tensor& t) {
  need(t.is_cuda() && t.layout() == at::kStrided && t.dim() == 2);
  Matrix m;
  m.type = t.scalar_type() == at::kBFloat16 ? QZ_BF16 : t.scalar_type() == at::kFloat ? QZ_F32 : -1;
  m.rows = t.size(0);
  m.cols = t.size(1);
  m.ld = m.rows <= 1 ? m.cols : t.stride(0);
  m.index = t.get_device();
  need(m.type >= 0 && (t.stride(1) == 1 || m.cols <= 1) && m.ld >= m.cols && m.index == c10::hip::current_device());
  m.p = t.data_ptr();
  return m;
}

int64_t pitch_of(int64_t cols) {
  need(cols >= 1 && cols <= QZ_I8_MAX_COLS);
  return (cols + 127) & ~int64_t{127};
}

// `rows` stored rows of `cols` columns.
void rows_of(PyObject* codes, PyObject* scales, int64_t rows, int64_t cols, int64_t index, const int8_t** c,
             const float** s) {
  const at::Tensor& tc = on(codes, index, at::kChar);
  const at::Tensor& ts = on(scales, index, at::kFloat);
  const int64_t pitch = pitch_of(cols);
  need(tc.is_contiguous() && ts.is_contiguous() && tc.dim() >= 1 && tc.size(-1) == pitch &&
       tc.numel() == pitch * rows && ts.numel() == rows);
  *c = static_cast<const int8_t*>(tc.data_ptr());
  *s = static_cast<const float*>(ts.data_ptr());
}

const uint8_t* zeros_of(PyObject* o, int64_t rows, int64_t index) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = on(o, index, at::kByte);
  need(t.is_contiguous() && t.numel() == rows);
  return static_cast<const uint8_t*>(t.data_ptr());
}

template <class T>
const T* vector(PyObject* o, int64_t n, int64_t index, at::ScalarType type) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = on(o, index, type);
  need(t.dim() == 1 && t.size(0) == n && t.is_contiguous());
  return static_cast<const T*>(t.data_ptr());
}

at::ScalarType out_type(PyObject* o) {
  if (o == Py_None) return at::kBFloat16;
  need(THPDtype_Check(o));
  const at::ScalarType t = reinterpret_cast<THPDtype*>(o)->scalar_type;
  need(t == at::kBFloat16 || t == at::kFloat);
  return t;
}

// (straight from the device's allocator: the dispatcher takes as long again)
at::Tensor make(at::IntArrayRef size, at::ScalarType type, int64_t index) {
  return at::Tensor(at::detail::empty_cuda(size, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(index)), std::nullopt));
}

hipStream_t stream_of(int64_t index) {
  return c10::hip::getCurrentHIPStream(static_cast<c10::DeviceIndex>(index)).stream();
}

int64_t whole(PyObject* o) {
  need(PyLong_CheckExact(o));
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Leave{};
  }
  return v;
}
int32_t whole32(PyObject* o) {
  const int64_t v = whole(o);
  need(v >= INT32_MIN && v <= INT32_MAX);
  return static_cast<int32_t>(v);
}

// The library's call, without the interpreter's lock.
template <class F>
void call(F&& f) {
  int status;
  Py_BEGIN_ALLOW_THREADS;
  status = f();
  Py_END_ALLOW_THREADS;
  need(status == QZ_OK);
}

// f's result, or None where it leaves the call to Python or anything throws.
template <class F>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, F&& f) {
  try {
    if (have == want && lib.moe) return f();
  } catch (...) {
    PyErr_Clear();
  }
  Py_RETURN_NONE;
}

PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {   // X, colf, sums, values
  return guarded(n, 4, [&] {
    const Matrix x = matrix(tensor(a[0]));
    const int64_t pitch = pitch_of(x.cols);
    const float* colf = vector<float>(a[1], x.cols, x.index, at::kFloat);
    const bool sums = a[2] == Py_True, values = a[3] == Py_True;
    need((sums || a[2] == Py_False) && (values || a[3] == Py_False));
    at::Tensor codes = make({x.rows, pitch}, at::kChar, x.index), scales = make({x.rows}, at::kFloat, x.index), s, v;
    if (sums) s = make({x.rows}, at::kInt, x.index);
    if (values) v = make({x.rows, x.cols}, x.type == QZ_BF16 ? at::kBFloat16 : at::kFloat, x.index);
    int8_t* const c = static_cast<int8_t*>(codes.data_ptr());
    float* const f = static_cast<float*>(scales.data_ptr());
    int32_t* const i = sums ? static_cast<int32_t*>(s.data_ptr()) : nullptr;
    void* const o = values ? v.data_ptr() : nullptr;
    const hipStream_t st = stream_of(x.index);
    call([&] { return lib.quantize(x.p, x.type, x.rows, x.cols, x.ld, colf, c, f, i, o, st); });
    PyObject* out = PyTuple_New(2 + sums + values);
    need(out);
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(std::move(codes)));
    PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(std::move(scales)));
    if (sums) PyTuple_SET_ITEM(out, 2, THPVariable_Wrap(std::move(s)));
    if (values) PyTuple_SET_ITEM(out, 2 + sums, THPVariable_Wrap(std::move(v)));
    return out;
  });
}

PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {   // X, codes, scales, zeros, colf, bias, out_dtype
  return guarded(n, 7, [&] {
    const Matrix x = matrix(tensor(a[0]));
    const at::Tensor& w = tensor(a[1]);
    need(w.dim() >= 1);
    const int64_t d_o = w.size(0);
    const int8_t* c;
    const float* s;
    rows_of(a[1], a[2], d_o, x.cols, x.index, &c, &s);
    const uint8_t* z = zeros_of(a[3], d_o, x.index);
    const float* colf = vector<float>(a[4], x.cols, x.index, at::kFloat);
    const float* bias = vector<float>(a[5], d_o, x.index, at::kFloat);
    const at::ScalarType type = out_type(a[6]);
    at::Tensor y = make({x.rows, d_o}, type, x.index), ws;
    const size_t bytes = lib.linear_workspace(x.rows, d_o, x.cols);
    if (bytes) ws = make({static_cast<int64_t>(bytes)}, at::kByte, x.index);
    void* const wp = bytes ? ws.data_ptr() : nullptr;
    void* const yp = y.data_ptr();
    const hipStream_t st = stream_of(x.index);
    call([&] {
      return lib.linear(x.p, x.type, x.rows, x.ld, colf, c, s, z, d_o, x.cols, bias, yp,
                        type == at::kFloat ? QZ_F32 : QZ_BF16, d_o, wp, bytes, st);
    });
    return THPVariable_Wrap(std::move(y));
  });
}

// xcodes, xscales, codes, scales, d_i, zeros, xsums, bias, out_dtype
PyObject* matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&] {
    const at::Tensor &x = tensor(a[0]), &w = tensor(a[2]);
    need(x.is_cuda() && x.dim() >= 1 && w.dim() >= 1 && x.get_device() == c10::hip::current_device());
    const int64_t index = x.get_device(), rows = x.size(0), d_o = w.size(0), d_i = whole(a[4]);
    const int8_t *xc, *c;
    const float *xs, *s;
    rows_of(a[0], a[1], rows, d_i, index, &xc, &xs);
    rows_of(a[2], a[3], d_o, d_i, index, &c, &s);
    const uint8_t* z = zeros_of(a[5], d_o, index);
    const int32_t* sums = vector<int32_t>(a[6], rows, index, at::kInt);
    need(!z || sums || rows == 0);
    const float* bias = vector<float>(a[7], d_o, index, at::kFloat);
    const at::ScalarType type = out_type(a[8]);
    at::Tensor y = make({rows, d_o}, type, index), ws;
    const size_t bytes = lib.matmul_workspace(rows, d_o, d_i);
    if (bytes) ws = make({static_cast<int64_t>(bytes)}, at::kByte, index);
    void* const wp = bytes ? ws.data_ptr() : nullptr;
    void* const yp = y.data_ptr();
    const hipStream_t st = stream_of(index);
    call([&] {
      return lib.matmul(xc, xs, sums, rows, c, s, z, d_o, d_i, bias, yp, type == at::kFloat ? QZ_F32 : QZ_BF16,
                        d_o, wp, bytes, st);
    });
    return THPVariable_Wrap(std::move(y));
  });
}

// logits, top_k, flags, bias, groups, top_groups, group_best, scale
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const Matrix x = matrix(tensor(a[0]));
    need(x.cols <= QZ_ROUTE_MAX_EXPERTS && (PyFloat_CheckExact(a[7]) || PyLong_CheckExact(a[7])));
    qz_router p{};
    p.struct_size = sizeof p;
    p.n_experts = static_cast<int32_t>(x.cols);
    p.top_k = whole32(a[1]);
    p.flags = static_cast<uint32_t>(whole32(a[2]));
    p.n_groups = whole32(a[4]);
    p.top_groups = whole32(a[5]);
    p.group_best = whole32(a[6]);
    const double scale = PyFloat_AsDouble(a[7]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      throw Leave{};
    }
    p.scale = static_cast<float>(scale);
    need(p.top_k >= 1 && p.top_k <= QZ_ROUTE_MAX_TOP_K);
    const float* bias = vector<float>(a[3], x.cols, x.index, at::kFloat);
    at::Tensor ids = make({x.rows, p.top_k}, at::kInt, x.index), w = make({x.rows, p.top_k}, at::kFloat, x.index);
    int32_t* const ip = static_cast<int32_t*>(ids.data_ptr());
    float* const wp = static_cast<float*>(w.data_ptr());
    const hipStream_t st = stream_of(x.index);
    call([&] { return lib.route(x.p, x.type, x.rows, x.ld, &p, bias, ip, wp, st); });
    PyObject* out = PyTuple_New(2);
    need(out);
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(std::move(ids)));
    PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(std::move(w)));
    return out;
  });
}

// X, ids, weights, gu_codes, gu_scales, dn_codes, dn_scales, gu_zeros, dn_zeros
PyObject* moe(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&] {
    const Matrix x = matrix(tensor(a[0]));
    const at::Tensor &ids = on(a[1], x.index, at::kInt), &weights = on(a[2], x.index, at::kFloat);
    need(ids.dim() == 2 && ids.size(0) == x.rows && weights.sizes() == ids.sizes() && ids.is_contiguous() &&
         weights.is_contiguous());
    const at::Tensor &gs = tensor(a[4]), &ds = tensor(a[6]);
    need(gs.dim() == 2 && gs.size(1) % 2 == 0 && ds.dim() == 2 && ds.size(0) == gs.size(0) && ds.size(1) == x.cols);
    const int64_t E = gs.size(0), f = gs.size(1) / 2, d = x.cols, k = ids.size(1);
    need(E >= 1 && E <= QZ_ROUTE_MAX_EXPERTS && k >= 1 && k <= QZ_ROUTE_MAX_TOP_K);
    const int8_t *gc, *dc;
    const float *gp, *dp;
    rows_of(a[3], a[4], E * 2 * f, d, x.index, &gc, &gp);
    rows_of(a[5], a[6], E * d, f, x.index, &dc, &dp);
    const uint8_t *gz = zeros_of(a[7], E * 2 * f, x.index), *dz = zeros_of(a[8], E * d, x.index);
    const size_t bytes = lib.moe_workspace(x.rows, d, f, static_cast<int32_t>(E), static_cast<int32_t>(k));
    at::Tensor y = make({x.rows, d}, at::kBFloat16, x.index), ws;
    if (bytes) ws = make({static_cast<int64_t>(bytes)}, at::kByte, x.index);
    void* const wp = bytes ? ws.data_ptr() : nullptr;
    void* const yp = y.data_ptr();
    const int32_t* const ip = static_cast<const int32_t*>(ids.data_ptr());
    const float* const pp = static_cast<const float*>(weights.data_ptr());
    const hipStream_t st = stream_of(x.index);
    call([&] {
      return lib.moe(x.p, x.type, x.rows, x.ld, d, f, static_cast<int32_t>(E), static_cast<int32_t>(k), ip, pp, gc,
                     gp, gz, dc, dp, dz, yp, wp, bytes, st);
    });
    return THPVariable_Wrap(std::move(y));
  });
}

// The library's ABI version and the addresses of its functions, in the order of `lib`.
PyObject* init(PyObject*, PyObject* args) {
  int abi;
  unsigned long long p[8];
  if (!PyArg_ParseTuple(args, "iKKKKKKKK", &abi, p, p + 1, p + 2, p + 3, p + 4, p + 5, p + 6, p + 7)) return nullptr;
  if (abi != QZ_ABI_VERSION)
    return PyErr_Format(PyExc_ImportError, "built for ABI version %d, and the library has %d", QZ_ABI_VERSION, abi);
  static_assert(sizeof lib == sizeof p);
  __builtin_memcpy(&lib, p, sizeof p);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"init", init, METH_VARARGS, nullptr},
    {"quantize", reinterpret_cast<PyCFunction>(quantize), METH_FASTCALL, nullptr},
    {"linear", reinterpret_cast<PyCFunction>(linear), METH_FASTCALL, nullptr},
    {"matmul", reinterpret_cast<PyCFunction>(matmul), METH_FASTCALL, nullptr},
    {"route", reinterpret_cast<PyCFunction>(route), METH_FASTCALL, nullptr},
    {"moe", reinterpret_cast<PyCFunction>(moe), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
