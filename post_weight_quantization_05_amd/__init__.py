"""Python binding of libqz, the gfx950 HIP library behind include/qz.h.

Argument marshalling only: tensors are allocated with PyTorch on the current CUDA
(HIP) device, their pointers and the current stream are passed through ctypes, and
every step of every solver runs in the library's kernels.  The functions carry the
C names; see include/qz.h for the operation each one performs and its citation.

Importing this package does not load the library; the first call does, and fails
loudly if libqz.so has not been built (there is no CPU fallback).
"""
from __future__ import annotations

import ctypes as C

from . import _lib
from ._lib import (QZ_ADMM_DUAL_NO_RESCALE, QZ_ADMM_REFRESH_FROM_Z, QZ_ADMM_REFRESH_UNCLAMPED,  # noqa: F401
                   QZ_ADMM_WARM_START, QZ_BF16, QZ_F32, QZ_GRID_CALLER, QZ_H_ACCUMULATE,
                   QZ_H_NO_FINALIZE, QZ_I8_MAX_COLS, QZ_MOE_RENORM, QZ_MX4_FLOOR, QZ_MX4_LEAST,
                   QZ_ROUTE_RENORM, QZ_ROUTE_SIGMOID, QzAdmm, QzGrid, QzMoe, QzRouter)


class QzError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        super().__init__(f"{_lib.STATUS_NAMES.get(status, status)}: {message}")


def lib():
    return _lib._lib or _lib.load()


def _check(status: int):
    if status != 0:
        raise QzError(status, lib().qz_last_error().decode(errors="replace"))


_torch_module = None


def _torch():
    """torch, imported on first use (the statement itself takes longer than a look at a name)."""
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream():
    torch = _torch()
    return C.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dtype_code(t):
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return _lib.QZ_BF16
    if t.dtype == torch.float32:
        return _lib.QZ_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def _dev(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _grid(bits, group, caller=False):
    return QzGrid(C.sizeof(QzGrid), int(bits), int(group), _lib.QZ_GRID_CALLER if caller else 0)


def _workspace(nbytes, device):
    torch = _torch()
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def qz_abi_version() -> int:
    return lib().qz_abi_version()


def qz_hessian_workspace(n, d_i, xt=_lib.QZ_BF16) -> int:
    return lib().qz_hessian_workspace(n, d_i, xt)


def qz_build_hessian(X, damp=0.01, flags=0, H=None, ws=None, scaled=False):
    """H = X^T X + lambda I (X [n x d_i] bf16 or fp32 on the GPU).  Returns
    dict(H, diag, sigma, lam, H_scaled) (tensors; lam is a 1-element tensor; H_scaled =
    Sigma H Sigma when scaled=True, else None)."""
    torch = _torch()
    _dev(X, "X")
    n, d = X.shape
    xt = _dtype_code(X)
    dev = X.device
    if H is None:
        H = torch.empty((d, d), dtype=torch.float32, device=dev)
    diag = torch.empty(d, dtype=torch.float32, device=dev)
    sigma = torch.empty(d, dtype=torch.float32, device=dev)
    lam = torch.empty(1, dtype=torch.float32, device=dev)
    Hs = torch.empty((d, d), dtype=torch.float32, device=dev) if scaled else None
    need = lib().qz_hessian_workspace(n, d, xt)
    if ws is None:
        ws = _workspace(need, dev)
    _check(lib().qz_build_hessian(_ptr(X), xt, n, d, float(damp), int(flags), _ptr(H), _ptr(diag),
                                  _ptr(sigma), _ptr(Hs), _ptr(lam), _ptr(ws), ws.numel(),
                                  _stream()))
    return dict(H=H, diag=diag, sigma=sigma, lam=lam, H_scaled=Hs)


def qz_rtn_workspace(d_o, d_i) -> int:
    return lib().qz_rtn_workspace(d_o, d_i)


def qz_rtn(W, bits, group, scales=None, zeros=None, ws=None):
    """Round-to-nearest codes on the grid fit from W (or the given grid)."""
    torch = _torch()
    _dev(W, "W")
    d_o, d_i = W.shape
    caller = scales is not None
    G = d_i // group if group > 0 and d_i % group == 0 else 0
    if not caller:
        scales = torch.empty((d_o, G), dtype=torch.float32, device=W.device)
        zeros = torch.empty((d_o, G), dtype=torch.uint8, device=W.device)
    codes = torch.empty((d_o, d_i), dtype=torch.uint8, device=W.device)
    if ws is None:
        ws = _workspace(lib().qz_rtn_workspace(d_o, d_i), W.device)
    g = _grid(bits, group, caller)
    _check(lib().qz_rtn(_ptr(W), _dtype_code(W), d_o, d_i, C.byref(g), _ptr(codes), _ptr(scales),
                        _ptr(zeros), _ptr(ws), ws.numel(), _stream()))
    return codes, scales, zeros


def qz_rtn_noalloc(W, bits, group, scales=None, zeros=None, codes=None):
    """qz_rtn without a workspace (the library's static per-GPU status word; calls that
    overlap on one GPU race on it).  Outputs may be passed in so that nothing is
    allocated here either."""
    torch = _torch()
    _dev(W, "W")
    d_o, d_i = W.shape
    caller = scales is not None
    G = d_i // group if group > 0 and d_i % group == 0 else 0
    if not caller:
        scales = torch.empty((d_o, G), dtype=torch.float32, device=W.device)
        zeros = torch.empty((d_o, G), dtype=torch.uint8, device=W.device)
    if codes is None:
        codes = torch.empty((d_o, d_i), dtype=torch.uint8, device=W.device)
    g = _grid(bits, group, caller)
    _check(lib().qz_rtn_noalloc(_ptr(W), _dtype_code(W), d_o, d_i, C.byref(g), _ptr(codes),
                                _ptr(scales), _ptr(zeros), _stream()))
    return codes, scales, zeros


def qz_gptq_workspace(d_o, d_i, B) -> int:
    return lib().qz_gptq_workspace(d_o, d_i, B)


def qz_gptq(H, W_hat, bits, group, B=128, perm=None, scales=None, zeros=None, ws=None):
    """GPTQ codes and grid for W_hat [d_o x d_i] given H [d_i x d_i]."""
    torch = _torch()
    _dev(H, "H")
    _dev(W_hat, "W_hat")
    d_o, d_i = W_hat.shape
    caller = scales is not None
    G = d_i // group if group > 0 and d_i % group == 0 else 0
    if not caller:
        scales = torch.empty((d_o, G), dtype=torch.float32, device=W_hat.device)
        zeros = torch.empty((d_o, G), dtype=torch.uint8, device=W_hat.device)
    codes = torch.empty((d_o, d_i), dtype=torch.uint8, device=W_hat.device)
    if perm is not None:
        perm = _dev(perm.to(torch.int32), "perm")
    if ws is None:
        ws = _workspace(lib().qz_gptq_workspace(d_o, d_i, B), W_hat.device)
    g = _grid(bits, group, caller)
    _check(lib().qz_gptq(_ptr(H), _ptr(W_hat), _dtype_code(W_hat), d_o, d_i, C.byref(g), int(B),
                         _ptr(perm), _ptr(codes), _ptr(scales), _ptr(zeros), _ptr(ws), ws.numel(),
                         _stream()))
    return codes, scales, zeros


def qz_gptq_noclip(H, W_hat, bits, group, B=128, perm=None, scales=None, zeros=None, ws=None):
    """GPTQ without clipping: int32 codes (may leave [0, 2^bits - 1]) and the grid."""
    torch = _torch()
    _dev(H, "H")
    _dev(W_hat, "W_hat")
    d_o, d_i = W_hat.shape
    caller = scales is not None
    G = d_i // group if group > 0 and d_i % group == 0 else 0
    if not caller:
        scales = torch.empty((d_o, G), dtype=torch.float32, device=W_hat.device)
        zeros = torch.empty((d_o, G), dtype=torch.uint8, device=W_hat.device)
    codes = torch.empty((d_o, d_i), dtype=torch.int32, device=W_hat.device)
    if perm is not None:
        perm = _dev(perm.to(torch.int32), "perm")
    if ws is None:
        ws = _workspace(lib().qz_gptq_workspace(d_o, d_i, B), W_hat.device)
    g = _grid(bits, group, caller)
    _check(lib().qz_gptq_noclip(_ptr(H), _ptr(W_hat), _dtype_code(W_hat), d_o, d_i, C.byref(g),
                                int(B), _ptr(perm), _ptr(codes), _ptr(scales), _ptr(zeros),
                                _ptr(ws), ws.numel(), _stream()))
    return codes, scales, zeros


def qz_order(H, kind, pivots=False, ws=None):
    """Quantization order for qz_gptq's perm: kind "act" or "min_pivot".  Returns perm
    (int32) or, with pivots=True (min_pivot only), (perm, LDL pivots fp64)."""
    torch = _torch()
    _dev(H, "H")
    d = H.shape[0]
    k = {"act": _lib.QZ_ORDER_ACT, "min_pivot": _lib.QZ_ORDER_MIN_PIVOT}[kind]
    perm = torch.empty(d, dtype=torch.int32, device=H.device)
    piv = torch.empty(d, dtype=torch.float64, device=H.device) if pivots else None
    if ws is None:
        ws = _workspace(lib().qz_order_workspace(d, k), H.device)
    _check(lib().qz_order(_ptr(H), d, k, _ptr(perm), _ptr(piv), _ptr(ws), ws.numel(), _stream()))
    return (perm, piv) if pivots else perm


def qz_error_bound(H, scales, group, perm=None, rows=False, ws=None):
    """Theorem 5 bound on the no-clip layer objective in order perm: the total (float)
    and, with rows=True, the per-row bounds (device fp64)."""
    torch = _torch()
    _dev(H, "H")
    _dev(scales, "scales")
    d_i = H.shape[0]
    d_o = scales.shape[0]
    if perm is not None:
        perm = _dev(perm.to(torch.int32), "perm")
    out = C.c_double(0.0)
    rb = torch.empty(max(d_o, 1), dtype=torch.float64, device=H.device)
    if ws is None:
        ws = _workspace(lib().qz_error_bound_workspace(d_o, d_i), H.device)
    _check(lib().qz_error_bound(_ptr(H), d_i, _ptr(perm), _ptr(scales), d_o, int(group), _ptr(rb),
                                C.byref(out), _ptr(ws), ws.numel(), _stream()))
    return (out.value, rb[:d_o]) if rows else out.value


def qz_admmq_prepare_workspace(d_i) -> int:
    return lib().qz_admmq_prepare_workspace(d_i)


def qz_admmq_prepare(H, ws=None):
    """(V, Lambda, sigma) with Sigma H Sigma = V diag(Lambda) V^T."""
    torch = _torch()
    _dev(H, "H")
    d = H.shape[0]
    V = torch.empty((d, d), dtype=torch.float32, device=H.device)
    lam = torch.empty(d, dtype=torch.float32, device=H.device)
    sigma = torch.empty(d, dtype=torch.float32, device=H.device)
    if ws is None:
        need = lib().qz_admmq_prepare_workspace(d)
        if need == 0:
            _check(-5)
        ws = _workspace(need, H.device)
    _check(lib().qz_admmq_prepare(_ptr(H), d, _ptr(V), _ptr(lam), _ptr(sigma), _ptr(ws), ws.numel(),
                                  _stream()))
    return V, lam, sigma


def qz_admmq_workspace(d_o, d_i, group, iters) -> int:
    return lib().qz_admmq_workspace(d_o, d_i, group, iters)


def qz_admmq(V, Lambda, sigma, W_hat, bits, group, iters, rho0, gamma, refresh_every=1, flags=0,
             t0=0, state=None, scales=None, zeros=None, ws=None, want_U=True):
    """ADMM-Q.  state: dict(codes, scales, zeros, U) to resume (sets QZ_ADMM_WARM_START;
    the tensors are updated in place).  Returns dict(codes, scales, zeros, U, residuals)."""
    torch = _torch()
    for t, nm in ((V, "V"), (Lambda, "Lambda"), (sigma, "sigma"), (W_hat, "W_hat")):
        _dev(t, nm)
    d_o, d_i = W_hat.shape
    dev = W_hat.device
    G = d_i // group if group > 0 and d_i % group == 0 else 0
    caller = scales is not None
    if state is not None:
        flags |= _lib.QZ_ADMM_WARM_START
        codes, scales, zeros, U = state["codes"], state["scales"], state["zeros"], state["U"]
    else:
        codes = torch.empty((d_o, d_i), dtype=torch.uint8, device=dev)
        if not caller:
            scales = torch.empty((d_o, G), dtype=torch.float32, device=dev)
            zeros = torch.empty((d_o, G), dtype=torch.uint8, device=dev)
        U = torch.empty((d_o, d_i), dtype=torch.float32, device=dev) if want_U else None
    res = torch.empty((max(iters, 1), 2), dtype=torch.float32, device=dev)
    if ws is None:
        ws = _workspace(lib().qz_admmq_workspace(d_o, d_i, group, iters), dev)
    g = _grid(bits, group, caller)
    p = QzAdmm(C.sizeof(QzAdmm), int(iters), float(rho0), float(gamma), int(refresh_every), int(flags),
               int(t0))
    _check(lib().qz_admmq(_ptr(V), _ptr(Lambda), _ptr(sigma), _ptr(W_hat), _dtype_code(W_hat), d_o,
                          d_i, C.byref(g), C.byref(p), _ptr(codes), _ptr(scales), _ptr(zeros),
                          _ptr(U), _ptr(res), _ptr(ws), ws.numel(), _stream()))
    return dict(codes=codes, scales=scales, zeros=zeros, U=U, residuals=res[:iters])


def qz_objective_workspace(d_o, d_i) -> int:
    return lib().qz_objective_workspace(d_o, d_i)


def qz_objective(H, W_hat, codes, scales, zeros, group, rows=False, ws=None):
    """f = 1/2 sum_r (q_r - w_r)^T H (q_r - w_r) for q = s (codes - z), codes uint8 or int32
    (no-clip GPTQ).  Returns the float (and, with rows=True, the per-row fp64 objectives as
    a device tensor)."""
    torch = _torch()
    for t, nm in ((H, "H"), (W_hat, "W_hat"), (codes, "codes"), (scales, "scales"), (zeros, "zeros")):
        _dev(t, nm)
    d_o, d_i = W_hat.shape
    if ws is None:
        ws = _workspace(lib().qz_objective_workspace(d_o, d_i), W_hat.device)
    row_f = torch.empty(d_o, dtype=torch.float64, device=W_hat.device) if rows else None
    out = C.c_double(0.0)
    fn = lib().qz_objective_i32 if codes.dtype == torch.int32 else lib().qz_objective
    _check(fn(_ptr(H), _ptr(W_hat), _dtype_code(W_hat), _ptr(codes), _ptr(scales), _ptr(zeros), d_o,
              d_i, int(group), _ptr(row_f), C.byref(out), _ptr(ws), ws.numel(), _stream()))
    return (out.value, row_f) if rows else out.value


def qz_local_search_workspace(d_o, d_i, group) -> int:
    return lib().qz_local_search_workspace(d_o, d_i, group)


def qz_local_search(H, W_hat, codes, scales, zeros, bits, group, max_steps, ws=None):
    """Pairwise-swap local search on the fixed grid; codes are updated in place.
    Returns (steps that moved, [moves accepted per step])."""
    for t, nm in ((H, "H"), (W_hat, "W_hat"), (codes, "codes"), (scales, "scales"), (zeros, "zeros")):
        _dev(t, nm)
    d_o, d_i = W_hat.shape
    if ws is None:
        ws = _workspace(lib().qz_local_search_workspace(d_o, d_i, group), W_hat.device)
    moves = (C.c_int32 * max(int(max_steps), 1))()
    steps = C.c_int32(0)
    g = _grid(bits, group, True)
    _check(lib().qz_local_search(_ptr(H), _ptr(W_hat), _dtype_code(W_hat), d_o, d_i, C.byref(g),
                                 _ptr(scales), _ptr(zeros), _ptr(codes), int(max_steps), moves,
                                 C.byref(steps), _ptr(ws), ws.numel(), _stream()))
    return steps.value, list(moves)[:steps.value + (1 if steps.value < max_steps else 0)]


def qz_packed_words(cols, bits) -> int:
    return lib().qz_packed_words(cols, bits)


def qz_pack(codes, bits):
    torch = _torch()
    _dev(codes, "codes")
    rows, cols = codes.shape
    out = torch.empty((rows, max(lib().qz_packed_words(cols, bits), 0)), dtype=torch.int32,
                      device=codes.device)
    _check(lib().qz_pack(_ptr(codes), rows, cols, int(bits), _ptr(out), _stream()))
    return out


def qz_unpack(words, cols, bits):
    torch = _torch()
    _dev(words, "words")
    rows = words.shape[0]
    out = torch.empty((rows, cols), dtype=torch.uint8, device=words.device)
    _check(lib().qz_unpack(_ptr(words), rows, cols, int(bits), _ptr(out), _stream()))
    return out


# ------------------------------------------------------------- microscaled 4-bit weights
# A call on a small matrix takes the GPU a few microseconds, so these functions ask torch for as
# little as they can: device indices instead of device objects, and the raw stream handle.
def _matrix(t, name):
    """Row stride of a 2-D GPU tensor with contiguous rows that do not overlap."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    rows, cols = t.shape
    ld, step = t.stride()
    if rows <= 1:      # the stride of a single row is of no meaning
        ld = cols
    if (step != 1 and cols > 1) or ld < cols:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return ld


def _mx4_pair(codes, scales, rows, cols, name, index):
    """Checks that codes and scales store `rows` rows of `cols` columns, on GPU `index`."""
    blocks = (cols + 31) >> 5
    u8 = _torch().uint8
    if codes.dtype is not u8 or scales.dtype is not u8:
        raise TypeError(f"{name}: codes and scales must be uint8")
    if codes.get_device() != index or scales.get_device() != index:
        raise ValueError(f"{name}: codes and scales must be on GPU {index}")
    if not (codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError(f"{name}: codes and scales must be contiguous")
    if codes.shape == (rows, 16 * blocks) and scales.shape == (rows, blocks):
        return
    if codes.shape[-1] != 16 * blocks or scales.shape[-1] != blocks \
            or codes.numel() != 16 * blocks * rows or scales.numel() != blocks * rows:
        raise ValueError(f"{name}: expected {rows} rows of {16 * blocks} code bytes and {blocks} factors")


def _vector(t, n, name, index):
    if t is None:
        return None
    if t.dtype is not _torch().float32:
        raise TypeError(f"{name} must be fp32")
    if t.get_device() != index or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous values on GPU {index}")
    return t.data_ptr()


def _scratch(ws, need, device):
    """(pointer, size) of a workspace of `need` bytes: the caller's, a new one, or none."""
    if ws is None:
        if need == 0:
            return None, 0, None
        ws = _workspace(need, device)
    elif ws.device != device or not ws.is_contiguous():
        raise ValueError("ws must be contiguous and on the inputs' GPU")
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


def _run(index, fn, *args):
    """fn(*args, stream) on the current stream of GPU `index`, with that GPU current."""
    cuda = _torch()._C
    if cuda._cuda_getDevice() == index:
        st = fn(*args, cuda._cuda_getCurrentRawStream(index))
    else:
        with _torch().cuda.device(index):
            st = fn(*args, cuda._cuda_getCurrentRawStream(index))
    if st != 0:
        _check(st)


def qz_mx4_blocks(cols) -> int:
    return lib().qz_mx4_blocks(cols)


def qz_mx4_quantize(W, rule="floor", colw=None, values=False):
    """Round a matrix (bf16 or fp32, contiguous rows) to MX4: (codes [rows x 16 G] uint8, scales
    [rows x G] uint8), and with values=True the numbers they stand for in W's dtype.  rule
    "floor", or "least" (the better of two factors per block under the column weights colw)."""
    torch = _torch()
    ld = _matrix(W, "W")
    wt = _dtype_code(W)
    rows, cols = W.shape
    if cols < 1:
        raise ValueError("W has no columns")
    if rule not in ("floor", "least"):
        raise ValueError(f"rule must be 'floor' or 'least', not {rule!r}")
    dev, blocks = W.device, (cols + 31) >> 5
    codes = W.new_empty((rows, 16 * blocks), dtype=torch.uint8)
    scales = codes.new_empty((rows, blocks))
    out = W.new_empty((rows, cols)) if values else None
    _run(dev.index, lib().qz_mx4_quantize, W.data_ptr(), wt, rows, cols, ld,
         _lib.QZ_MX4_LEAST if rule == "least" else _lib.QZ_MX4_FLOOR,
         _vector(colw, cols, "colw", dev.index), codes.data_ptr(), scales.data_ptr(),
         out.data_ptr() if values else None)
    return (codes, scales, out) if values else (codes, scales)


def qz_mx4_unpack(codes, scales, cols):
    """(codes int32, scales fp32, zeros uint8): the stored matrix in qz_objective's form (group
    size 32)."""
    torch = _torch()
    _dev(codes, "codes")
    rows, dev = codes.shape[0], codes.device
    _mx4_pair(codes, scales, rows, cols, "matrix", dev.index)
    out = torch.empty((rows, cols), dtype=torch.int32, device=dev)
    s = torch.empty(scales.shape, dtype=torch.float32, device=dev)
    z = torch.empty(scales.shape, dtype=torch.uint8, device=dev)
    _run(dev.index, lib().qz_mx4_unpack, codes.data_ptr(), scales.data_ptr(), rows, cols,
         out.data_ptr(), s.data_ptr(), z.data_ptr())
    return out, s, z


def _product_out(out, like, n, d_o, dtype, device):
    """(out, its row stride, its dtype code) for a product's result, on the GPU of `like`."""
    torch = _torch()
    if out is None:
        if dtype is None or dtype is torch.bfloat16:
            if like.dtype is torch.bfloat16:
                return like.new_empty((n, d_o)), d_o, _lib.QZ_BF16
            return like.new_empty((n, d_o), dtype=torch.bfloat16), d_o, _lib.QZ_BF16
        if dtype is not torch.float32:
            raise TypeError(f"unsupported dtype {dtype} (bf16 or fp32)")
        return like.new_empty((n, d_o), dtype=dtype), d_o, _lib.QZ_F32
    if tuple(out.shape) != (n, d_o) or (dtype is not None and out.dtype != dtype):
        raise ValueError(f"out must be [{n} x {d_o}]" + (f" {dtype}" if dtype is not None else ""))
    if out.device != device:
        raise ValueError(f"out must be on {device}")
    return out, _matrix(out, "out"), _dtype_code(out)


def qz_mx4_linear_workspace(n, d_o, d_i) -> int:
    """Bytes that suffice for any address and row stride of X."""
    return lib().qz_mx4_linear_workspace(None, n, 0, d_o, d_i)


def qz_mx4_linear(X, codes, scales, bias=None, out_dtype=None, out=None, ws=None):
    """Y = X W^T + bias for X bf16 [n x d_i] (contiguous rows) and W [d_o x d_i] in MX4.  Y is
    out_dtype (bf16 or fp32; default bf16), or `out` is written."""
    L = lib()
    ldx = _matrix(X, "X")
    if _dtype_code(X) != _lib.QZ_BF16:
        raise TypeError("X must be bf16")
    (n, d_i), d_o, dev, x = X.shape, codes.shape[0], X.device, X.data_ptr()
    index = dev.index
    _mx4_pair(codes, scales, d_o, d_i, "W", index)
    out, ldy, yt = _product_out(out, codes, n, d_o, out_dtype, dev)
    wp, wn, ws = _scratch(ws, L.qz_mx4_linear_workspace(x, n, ldx, d_o, d_i), dev)
    _run(index, L.qz_mx4_linear, x, _lib.QZ_BF16, n, ldx, codes.data_ptr(), scales.data_ptr(), d_o,
         d_i, _vector(bias, d_o, "bias", index), out.data_ptr(), yt, ldy, wp, wn)
    return out


def qz_mx4_matmul_workspace(n, d_o, d_i) -> int:
    return lib().qz_mx4_matmul_workspace(n, d_o, d_i)


def qz_mx4_matmul(xcodes, xscales, codes, scales, d_i, bias=None, out_dtype=None, out=None, ws=None):
    """Y = X W^T + bias with X [n x d_i] and W [d_o x d_i] both in MX4."""
    L = lib()
    _dev(xcodes, "X codes")
    n, d_o, dev = xcodes.shape[0], codes.shape[0], xcodes.device
    index = dev.index
    _mx4_pair(xcodes, xscales, n, d_i, "X", index)
    _mx4_pair(codes, scales, d_o, d_i, "W", index)
    out, ldy, yt = _product_out(out, codes, n, d_o, out_dtype, dev)
    wp, wn, ws = _scratch(ws, L.qz_mx4_matmul_workspace(n, d_o, d_i), dev)
    _run(index, L.qz_mx4_matmul, xcodes.data_ptr(), xscales.data_ptr(), n, codes.data_ptr(),
         scales.data_ptr(), d_o, d_i, _vector(bias, d_o, "bias", index), out.data_ptr(), yt, ldy,
         wp, wn)
    return out


def _moe_params(n_experts, top_k, renorm):
    n_experts, top_k = int(n_experts), int(top_k)
    if abs(n_experts) >> 31 or abs(top_k) >> 31:      # ctypes would cut them to 32 bits
        raise ValueError("the number of experts and top_k must fit 32 bits")
    return QzMoe(C.sizeof(QzMoe), n_experts, top_k, _lib.QZ_MOE_RENORM if renorm else 0)


def qz_mx4_moe_workspace(n, d, f, n_experts, top_k) -> int:
    return lib().qz_mx4_moe_workspace(n, d, f, C.byref(_moe_params(n_experts, top_k, False)))


def qz_mx4_moe(X, router, gu_codes, gu_scales, dn_codes, dn_scales, top_k, renorm=True,
               routing=False, ws=None):
    """The routed expert layer for few tokens: X bf16 [n x d], router [E x d] (bf16 or fp32),
    gate and up weights [E x 2f x d] and down weights [E x d x f] in MX4.  Returns Y bf16
    [n x d], and with routing=True also (ids int32, weights fp32) [n x top_k]."""
    torch, L = _torch(), lib()
    ldx = _matrix(X, "X")
    if _dtype_code(X) != _lib.QZ_BF16:
        raise TypeError("X must be bf16")
    (n, d), dev, k = X.shape, X.device, int(top_k)
    index = dev.index
    if router.dim() != 2 or router.shape[1] != d or gu_codes.dim() != 3 or gu_codes.shape[1] % 2:
        raise ValueError("router must be [E x d], the gate and up weights [E x 2f x d]")
    if router.get_device() != index or not router.is_contiguous():
        raise ValueError("router must be contiguous and on the inputs' GPU")
    E, f = router.shape[0], gu_codes.shape[1] // 2
    if gu_codes.shape[0] != E or dn_codes.dim() != 3 or dn_codes.shape[0] != E or dn_codes.shape[1] != d:
        raise ValueError("the experts' weights must be [E x 2f x d] and [E x d x f]")
    _mx4_pair(gu_codes, gu_scales, E * 2 * f, d, "gate and up weights", index)
    _mx4_pair(dn_codes, dn_scales, E * d, f, "down weights", index)
    p = C.byref(_moe_params(E, k, renorm))
    wp, wn, ws = _scratch(ws, L.qz_mx4_moe_workspace(n, d, f, p), dev)
    y = torch.empty((n, d), dtype=torch.bfloat16, device=dev)
    if routing and k > 0:
        ids = torch.empty((n, k), dtype=torch.int32, device=dev)
        w = torch.empty((n, k), dtype=torch.float32, device=dev)
        ip, kp = ids.data_ptr(), w.data_ptr()
    else:
        ip = kp = None
    _run(index, L.qz_mx4_moe, X.data_ptr(), _lib.QZ_BF16, n, ldx, d, f, p, router.data_ptr(),
         _dtype_code(router), gu_codes.data_ptr(), gu_scales.data_ptr(), dn_codes.data_ptr(),
         dn_scales.data_ptr(), y.data_ptr(), ip, kp, wp, wn)
    return (y, ids, w) if routing else y


# ------------------------------------------------------------------ 8-bit integer products
# The ordinary call goes through _lib.binding (csrc/binding.cpp), which returns None for one that it leaves
# to the code here: another GPU, a caller's output or workspace, or an argument that has to be refused.
def qz_i8_pitch(cols) -> int:
    return lib().qz_i8_pitch(cols)


def _i8_rows(codes, scales, rows, cols, name, index):
    """Checks that codes and scales store `rows` rows of `cols` columns, on GPU `index`."""
    torch = _torch()
    if not 1 <= cols <= QZ_I8_MAX_COLS:
        raise ValueError(f"{name} must have 1 to {QZ_I8_MAX_COLS} columns")
    if codes.dtype is not torch.int8 or scales.dtype is not torch.float32:
        raise TypeError(f"{name}: codes must be int8 and scales fp32")
    if codes.get_device() != index or scales.get_device() != index:
        raise ValueError(f"{name}: codes and scales must be on GPU {index}")
    if not (codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError(f"{name}: codes and scales must be contiguous")
    pitch = (cols + 127) & ~127
    if codes.numel() != pitch * rows or scales.numel() != rows or codes.shape[-1] != pitch:
        raise ValueError(f"{name}: expected {rows} rows of {pitch} codes and {rows} scales")


def _i8_zeros(t, rows, name, index):
    if t is None:
        return None
    if t.dtype is not _torch().uint8:
        raise TypeError(f"{name}: zeros must be uint8")
    if t.get_device() != index or t.numel() != rows or not t.is_contiguous():
        raise ValueError(f"{name}: zeros must be {rows} contiguous values on GPU {index}")
    return t.data_ptr()


def qz_i8_quantize(X, colf=None, sums=False, values=False):
    """Rows of a matrix (bf16 or fp32, contiguous rows), times the column factors colf, to int8 with a
    scale each: (codes int8 [rows x pitch], scales fp32 [rows]), then with sums=True the rows' sums of
    codes (int32), and with values=True the numbers the codes stand for in X's dtype."""
    if _lib.binding is not None:
        r = _lib.binding.quantize(X, colf, sums, values)
        if r is not None:
            return r
    torch = _torch()
    ld = _matrix(X, "X")
    xt = _dtype_code(X)
    rows, cols = X.shape
    if not 1 <= cols <= QZ_I8_MAX_COLS:
        raise ValueError(f"X must have 1 to {QZ_I8_MAX_COLS} columns")
    index = X.device.index
    codes = X.new_empty((rows, (cols + 127) & ~127), dtype=torch.int8)
    scales = X.new_empty((rows,)) if xt == _lib.QZ_F32 else X.new_empty((rows,), dtype=torch.float32)
    total = X.new_empty((rows,), dtype=torch.int32) if sums else None
    out = X.new_empty((rows, cols)) if values else None
    _run(index, lib().qz_i8_quantize, X.data_ptr(), xt, rows, cols, ld, _vector(colf, cols, "colf", index),
         codes.data_ptr(), scales.data_ptr(), total.data_ptr() if sums else None,
         out.data_ptr() if values else None)
    return (codes, scales) + ((total,) if sums else ()) + ((out,) if values else ())


def qz_i8_pack(codes):
    """The solvers' codes (uint8 [rows x cols]) as int8 codes less 128, in padded rows."""
    torch = _torch()
    _dev(codes, "codes")
    if codes.dtype is not torch.uint8 or codes.dim() != 2:
        raise TypeError("codes must be a uint8 matrix")
    rows, cols = codes.shape
    if not 1 <= cols <= QZ_I8_MAX_COLS:
        raise ValueError(f"codes must have 1 to {QZ_I8_MAX_COLS} columns")
    out = codes.new_empty((rows, (cols + 127) & ~127), dtype=torch.int8)
    _run(codes.device.index, lib().qz_i8_pack, codes.data_ptr(), rows, cols, out.data_ptr())
    return out


def qz_i8_unpack(codes, cols):
    """The int8 codes' uint8 form (code + 128), [rows x cols]."""
    torch = _torch()
    _dev(codes, "codes")
    if codes.dtype is not torch.int8 or codes.dim() != 2:
        raise TypeError("codes must be an int8 matrix")
    if not 1 <= cols <= QZ_I8_MAX_COLS or codes.shape[1] != (cols + 127) & ~127:
        raise ValueError(f"rows of {cols} columns do not have {codes.shape[1]} codes")
    out = codes.new_empty((codes.shape[0], cols), dtype=torch.uint8)
    _run(codes.device.index, lib().qz_i8_unpack, codes.data_ptr(), codes.shape[0], cols, out.data_ptr())
    return out


def qz_i8_matmul_workspace(n, d_o, d_i) -> int:
    return lib().qz_i8_matmul_workspace(n, d_o, d_i)


def qz_i8_matmul(xcodes, xscales, codes, scales, d_i, zeros=None, xsums=None, bias=None,
                 out_dtype=None, out=None, ws=None):
    """Y = X W^T + bias with X [n x d_i] and W [d_o x d_i] both as int8 rows.  zeros (the solvers'
    zero points of W, uint8 [d_o]) needs xsums, the row sums of X.  Y is out_dtype (bf16 or fp32;
    default bf16), or `out` is written."""
    if out is None and ws is None and _lib.binding is not None:
        r = _lib.binding.matmul(xcodes, xscales, codes, scales, d_i, zeros, xsums, bias, out_dtype)
        if r is not None:
            return r
    L = lib()
    _dev(xcodes, "X codes")
    n, d_o, dev = xcodes.shape[0], codes.shape[0], xcodes.device
    index = dev.index
    _i8_rows(xcodes, xscales, n, d_i, "X", index)
    _i8_rows(codes, scales, d_o, d_i, "W", index)
    zp = _i8_zeros(zeros, d_o, "W", index)
    if xsums is not None:
        if xsums.dtype is not _torch().int32:
            raise TypeError("xsums must be int32")
        if xsums.get_device() != index or xsums.shape != (n,) or not xsums.is_contiguous():
            raise ValueError(f"xsums must be {n} contiguous values on GPU {index}")
    elif zp is not None and n and d_o:
        raise ValueError("zeros need xsums, the row sums of X")
    out, ldy, yt = _product_out(out, codes, n, d_o, out_dtype, dev)
    wp, wn, ws = _scratch(ws, L.qz_i8_matmul_workspace(n, d_o, d_i), dev)
    _run(index, L.qz_i8_matmul, xcodes.data_ptr(), xscales.data_ptr(),
         None if xsums is None else xsums.data_ptr(), n, codes.data_ptr(), scales.data_ptr(), zp, d_o,
         d_i, _vector(bias, d_o, "bias", index), out.data_ptr(), yt, ldy, wp, wn)
    return out


def qz_i8_linear_workspace(n, d_o, d_i) -> int:
    return lib().qz_i8_linear_workspace(n, d_o, d_i)


def qz_i8_linear(X, codes, scales, zeros=None, colf=None, bias=None, out_dtype=None, out=None, ws=None):
    """Y = Q(X) W^T + bias: X (bf16 or fp32 [n x d_i], contiguous rows), times the column factors
    colf, is quantized per row in the same call; W [d_o x d_i] as int8 rows with zeros or without."""
    if out is None and ws is None and _lib.binding is not None:
        r = _lib.binding.linear(X, codes, scales, zeros, colf, bias, out_dtype)
        if r is not None:
            return r
    L = lib()
    ldx = _matrix(X, "X")
    xt = _dtype_code(X)
    (n, d_i), d_o, dev = X.shape, codes.shape[0], X.device
    index = dev.index
    _i8_rows(codes, scales, d_o, d_i, "W", index)
    out, ldy, yt = _product_out(out, X if xt == _lib.QZ_BF16 else codes, n, d_o, out_dtype, dev)
    wp, wn, ws = _scratch(ws, L.qz_i8_linear_workspace(n, d_o, d_i), dev)
    _run(index, L.qz_i8_linear, X.data_ptr(), xt, n, ldx, _vector(colf, d_i, "colf", index),
         codes.data_ptr(), scales.data_ptr(), _i8_zeros(zeros, d_o, "W", index), d_o, d_i,
         _vector(bias, d_o, "bias", index), out.data_ptr(), yt, ldy, wp, wn)
    return out


def _int32(v, name):
    v = int(v)
    if not -2 ** 31 <= v < 2 ** 31:      # ctypes would cut it to 32 bits
        raise ValueError(f"{name} must fit 32 bits")
    return v


def qz_route(logits, top_k, scores="softmax", bias=None, groups=1, top_groups=1, group_best=1,
             renorm=True, scale=1.0):
    """(ids int32, weights fp32) [n x top_k]: the experts of each token from the router's logits (bf16
    or fp32 [n x E], contiguous rows).  scores "softmax" or "sigmoid"; bias fp32 [E] moves the choice
    alone; of `groups` groups the best top_groups stay, each counted by the sum of its group_best
    (1 or 2) largest choices; weights divided by their sum with renorm, times scale."""
    if scores not in ("softmax", "sigmoid"):
        raise ValueError(f"scores must be 'softmax' or 'sigmoid', not {scores!r}")
    flags = (_lib.QZ_ROUTE_SIGMOID if scores == "sigmoid" else 0) | (_lib.QZ_ROUTE_RENORM if renorm else 0)
    if _lib.binding is not None:
        r = _lib.binding.route(logits, top_k, flags, bias, groups, top_groups, group_best, scale)
        if r is not None:
            return r
    torch = _torch()
    ld = _matrix(logits, "logits")
    lt = _dtype_code(logits)
    n, E = logits.shape
    k, index = _int32(top_k, "top_k"), logits.device.index
    p = QzRouter(C.sizeof(QzRouter), _int32(E, "the number of experts"), k, _int32(groups, "groups"),
                 _int32(top_groups, "top_groups"), _int32(group_best, "group_best"), flags, scale)
    ids = logits.new_empty((n, k if k > 0 else 0), dtype=torch.int32)
    w = logits.new_empty(ids.shape, dtype=torch.float32)
    _run(index, lib().qz_route, logits.data_ptr(), lt, n, ld, C.byref(p), _vector(bias, E, "bias", index),
         ids.data_ptr(), w.data_ptr())
    return ids, w


def qz_i8_moe_workspace(n, d, f, n_experts, top_k) -> int:
    return lib().qz_i8_moe_workspace(n, d, f, _int32(n_experts, "the number of experts"), _int32(top_k, "top_k"))


def qz_i8_moe(X, ids, weights, gu_codes, gu_scales, dn_codes, dn_scales, gu_zeros=None, dn_zeros=None,
              ws=None):
    """The routed expert layer on int8 weights: X (bf16 or fp32 [n x d]), ids (int32) and weights (fp32)
    [n x top_k] as qz_route returns them, gate and up weights [E x 2f x d] and down weights [E x d x f]
    as int8 rows with zeros or without.  Returns Y bf16 [n x d]; ids outside [0, E) are skipped."""
    if ws is None and _lib.binding is not None:
        r = _lib.binding.moe(X, ids, weights, gu_codes, gu_scales, dn_codes, dn_scales, gu_zeros, dn_zeros)
        if r is not None:
            return r
    torch, L = _torch(), lib()
    ldx = _matrix(X, "X")
    xt = _dtype_code(X)
    (n, d), dev = X.shape, X.device
    index = dev.index
    if gu_scales.dim() != 2 or gu_scales.shape[1] % 2 or dn_scales.dim() != 2:
        raise ValueError("the scales must be [E x 2f] and [E x d]")
    E, f = gu_scales.shape[0], gu_scales.shape[1] // 2
    if dn_scales.shape != (E, d):
        raise ValueError("the down weights must be [E x d x f]")
    _i8_rows(gu_codes, gu_scales, E * 2 * f, d, "gate and up weights", index)
    _i8_rows(dn_codes, dn_scales, E * d, f, "down weights", index)
    if ids.dtype is not torch.int32 or weights.dtype is not torch.float32:
        raise TypeError("ids must be int32 and weights fp32")
    if ids.dim() != 2 or ids.shape[0] != n or weights.shape != ids.shape:
        raise ValueError(f"ids and weights must be [{n} x top_k]")
    if ids.get_device() != index or weights.get_device() != index \
            or not (ids.is_contiguous() and weights.is_contiguous()):
        raise ValueError(f"ids and weights must be contiguous and on GPU {index}")
    k = ids.shape[1]
    wp, wn, ws = _scratch(ws, L.qz_i8_moe_workspace(n, d, f, E, k), dev)
    y = X.new_empty((n, d), dtype=torch.bfloat16)
    _run(index, L.qz_i8_moe, X.data_ptr(), xt, n, ldx, d, f, E, k, ids.data_ptr(), weights.data_ptr(),
         gu_codes.data_ptr(), gu_scales.data_ptr(), _i8_zeros(gu_zeros, E * 2 * f, "gate and up weights", index),
         dn_codes.data_ptr(), dn_scales.data_ptr(), _i8_zeros(dn_zeros, E * d, "down weights", index),
         y.data_ptr(), wp, wn)
    return y


def qz_timing_enable(on=True):
    _check(lib().qz_timing_enable(1 if on else 0))


def qz_timing_read(reset=True):
    """{kind name: (launches, total_ms)} of the launches recorded while timing was on."""
    n = 32
    launches = (C.c_int64 * n)()
    total = (C.c_double * n)()
    k = lib().qz_timing_read(launches, total, n, 1 if reset else 0)
    if k < 0:
        _check(k)
    return {lib().qz_timing_kind_name(i).decode(): (launches[i], total[i]) for i in range(min(k, n))
            if launches[i] > 0}


def qz_last_error() -> str:
    return lib().qz_last_error().decode(errors="replace")
