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
                   QZ_H_NO_FINALIZE, QZ_MOE_RENORM, QZ_MX4_FLOOR, QZ_MX4_LEAST, QzAdmm, QzGrid,
                   QzMoe)


class QzError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        super().__init__(f"{_lib.STATUS_NAMES.get(status, status)}: {message}")


def lib():
    return _lib.load()


def _check(status: int):
    if status != 0:
        raise QzError(status, lib().qz_last_error().decode(errors="replace"))


def _torch():
    import torch
    return torch


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
def _rows(t, name, dtypes):
    """A 2-D GPU tensor of one of `dtypes` whose rows are contiguous: (pointer, row stride)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    if t.dim() != 2 or t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must be a matrix with contiguous rows")
    if t.shape[0] <= 1:   # the stride of a single row is of no meaning
        return t.data_ptr(), t.shape[1]
    if t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}: rows overlap")
    return t.data_ptr(), t.stride(0)


def _mx4_pair(codes, scales, rows, cols, name, device):
    """Checks that codes and scales store matrices of the given total rows and columns."""
    torch = _torch()
    blocks = -(-cols // 32)
    for t, width, what in ((codes, 16 * blocks, "codes"), (scales, blocks, "scales")):
        if t.dtype != torch.uint8:
            raise TypeError(f"{name} {what} must be uint8")
        if t.device != device or not t.is_contiguous():
            raise ValueError(f"{name} {what} must be contiguous and on {device}")
        if t.numel() != rows * width or t.shape[-1] != width:
            raise ValueError(f"{name} {what}: expected {rows} rows of {width} bytes")


def _on(device, *others):
    """The raw current stream of `device`, where all `others` (or None) have to live too.  The
    call itself runs with that device current."""
    torch = _torch()
    for t in others:
        if t is not None and t.device != device:
            raise ValueError(f"tensors on {t.device} and {device} in one call")
    return torch.cuda.current_stream(device).cuda_stream


def _call(device, fn, *args):
    torch = _torch()
    if torch.cuda.current_device() == device.index:
        _check(fn(*args))
    else:
        with torch.cuda.device(device):
            _check(fn(*args))


def _vector(t, n, name, device):
    if t is None:
        return None
    if t.dtype != _torch().float32:
        raise TypeError(f"{name} must be fp32")
    if t.device != device or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous values on {device}")
    return t.data_ptr()


def qz_mx4_blocks(cols) -> int:
    return lib().qz_mx4_blocks(cols)


def qz_mx4_quantize(W, rule="floor", colw=None, values=False):
    """Round a matrix (bf16 or fp32, contiguous rows) to MX4: (codes [rows x 16 G] uint8, scales
    [rows x G] uint8), and with values=True the numbers they stand for in W's dtype.  rule
    "floor", or "least" (the better of two factors per block under the column weights colw)."""
    torch = _torch()
    ptr, ld = _rows(W, "W", (torch.bfloat16, torch.float32))
    rows, cols = W.shape
    if cols < 1:
        raise ValueError("W has no columns")
    k = {"floor": _lib.QZ_MX4_FLOOR, "least": _lib.QZ_MX4_LEAST}[rule]
    dev, blocks = W.device, -(-cols // 32)
    stream = _on(dev)
    codes = torch.empty((rows, 16 * blocks), dtype=torch.uint8, device=dev)
    scales = torch.empty((rows, blocks), dtype=torch.uint8, device=dev)
    out = torch.empty((rows, cols), dtype=W.dtype, device=dev) if values else None
    _call(dev, lib().qz_mx4_quantize, ptr, _dtype_code(W), rows, cols, ld, k,
          _vector(colw, cols, "colw", dev), codes.data_ptr(), scales.data_ptr(),
          out.data_ptr() if values else None, stream)
    return (codes, scales, out) if values else (codes, scales)


def qz_mx4_unpack(codes, scales, cols):
    """(codes int32, scales fp32, zeros uint8): the stored matrix in qz_objective's form (group
    size 32)."""
    torch = _torch()
    _dev(codes, "codes")
    rows, dev = codes.shape[0], codes.device
    _mx4_pair(codes, scales, rows, cols, "MX4", dev)
    out = torch.empty((rows, cols), dtype=torch.int32, device=dev)
    s = torch.empty(scales.shape, dtype=torch.float32, device=dev)
    z = torch.empty(scales.shape, dtype=torch.uint8, device=dev)
    _call(dev, lib().qz_mx4_unpack, codes.data_ptr(), scales.data_ptr(), rows, cols, out.data_ptr(),
          s.data_ptr(), z.data_ptr(), _on(dev))
    return out, s, z


def _product_out(out, n, d_o, dtype, device):
    torch = _torch()
    if out is None:
        out = torch.empty((n, d_o), dtype=dtype or torch.bfloat16, device=device)
    elif tuple(out.shape) != (n, d_o) or (dtype is not None and out.dtype != dtype):
        raise ValueError(f"out must be [{n} x {d_o}]" + (f" {dtype}" if dtype is not None else ""))
    ptr, ld = _rows(out, "out", (torch.bfloat16, torch.float32))
    return out, ptr, max(ld, d_o)


def qz_mx4_linear_workspace(n, d_o, d_i) -> int:
    return lib().qz_mx4_linear_workspace(n, d_o, d_i)


def qz_mx4_linear(X, codes, scales, bias=None, out_dtype=None, out=None, ws=None):
    """Y = X W^T + bias for X bf16 [n x d_i] (contiguous rows) and W [d_o x d_i] in MX4.  Y is
    out_dtype (bf16 or fp32; default bf16), or `out` is written."""
    torch = _torch()
    ptr, ldx = _rows(X, "X", (torch.bfloat16,))
    (n, d_i), d_o, dev = X.shape, codes.shape[0], X.device
    _mx4_pair(codes, scales, d_o, d_i, "W", dev)
    stream = _on(dev, out, ws)
    out, yp, ldy = _product_out(out, n, d_o, out_dtype, dev)
    if ws is None:
        ws = _workspace(lib().qz_mx4_linear_workspace(n, d_o, d_i), dev)
    _call(dev, lib().qz_mx4_linear, ptr, _lib.QZ_BF16, n, ldx, codes.data_ptr(), scales.data_ptr(),
          d_o, d_i, _vector(bias, d_o, "bias", dev), yp, _dtype_code(out), ldy, ws.data_ptr(),
          ws.numel(), stream)
    return out


def qz_mx4_matmul_workspace(n, d_o, d_i) -> int:
    return lib().qz_mx4_matmul_workspace(n, d_o, d_i)


def qz_mx4_matmul(xcodes, xscales, codes, scales, d_i, bias=None, out_dtype=None, out=None, ws=None):
    """Y = X W^T + bias with X [n x d_i] and W [d_o x d_i] both in MX4."""
    _dev(xcodes, "X codes")
    n, d_o, dev = xcodes.shape[0], codes.shape[0], xcodes.device
    _mx4_pair(xcodes, xscales, n, d_i, "X", dev)
    _mx4_pair(codes, scales, d_o, d_i, "W", dev)
    stream = _on(dev, out, ws)
    out, yp, ldy = _product_out(out, n, d_o, out_dtype, dev)
    if ws is None:
        ws = _workspace(lib().qz_mx4_matmul_workspace(n, d_o, d_i), dev)
    _call(dev, lib().qz_mx4_matmul, xcodes.data_ptr(), xscales.data_ptr(), n, codes.data_ptr(),
          scales.data_ptr(), d_o, d_i, _vector(bias, d_o, "bias", dev), yp, _dtype_code(out), ldy,
          ws.data_ptr(), ws.numel(), stream)
    return out


def _moe_params(n_experts, top_k, renorm):
    return QzMoe(C.sizeof(QzMoe), int(n_experts), int(top_k), _lib.QZ_MOE_RENORM if renorm else 0)


def qz_mx4_moe_workspace(n, d, f, n_experts, top_k) -> int:
    return lib().qz_mx4_moe_workspace(n, d, f, C.byref(_moe_params(n_experts, top_k, False)))


def qz_mx4_moe(X, router, gu_codes, gu_scales, dn_codes, dn_scales, top_k, renorm=True,
               routing=False, ws=None):
    """The routed expert layer for few tokens: X bf16 [n x d], router [E x d] (bf16 or fp32),
    gate and up weights [E x 2f x d] and down weights [E x d x f] in MX4.  Returns Y bf16
    [n x d], and with routing=True also (ids int32, weights fp32) [n x top_k]."""
    torch = _torch()
    ptr, ldx = _rows(X, "X", (torch.bfloat16,))
    (n, d), dev = X.shape, X.device
    _dev(router, "router")
    if router.dim() != 2 or router.shape[1] != d or gu_codes.dim() != 3 or gu_codes.shape[1] % 2:
        raise ValueError("router must be [E x d], the gate and up weights [E x 2f x d]")
    E, f = router.shape[0], gu_codes.shape[1] // 2
    if gu_codes.shape[0] != E or tuple(dn_codes.shape[:2]) != (E, d):
        raise ValueError("the experts' weights must be [E x 2f x d] and [E x d x f]")
    _mx4_pair(gu_codes, gu_scales, E * 2 * f, d, "gate and up", dev)
    _mx4_pair(dn_codes, dn_scales, E * d, f, "down", dev)
    stream = _on(dev, router, ws)
    p = _moe_params(E, top_k, renorm)
    if ws is None:
        ws = _workspace(lib().qz_mx4_moe_workspace(n, d, f, C.byref(p)), dev)
    k = max(int(top_k), 0)
    y = torch.empty((n, d), dtype=torch.bfloat16, device=dev)
    ids = torch.empty((n, k), dtype=torch.int32, device=dev) if routing else None
    w = torch.empty((n, k), dtype=torch.float32, device=dev) if routing else None
    _call(dev, lib().qz_mx4_moe, ptr, _lib.QZ_BF16, n, ldx, d, f, C.byref(p), router.data_ptr(),
          _dtype_code(router), gu_codes.data_ptr(), gu_scales.data_ptr(), dn_codes.data_ptr(),
          dn_scales.data_ptr(), y.data_ptr(), ids.data_ptr() if routing else None,
          w.data_ptr() if routing else None, ws.data_ptr(), ws.numel(), stream)
    return (y, ids, w) if routing else y


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
