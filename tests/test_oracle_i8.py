"""CPU: the 8-bit integer oracle against values worked out by hand, and the refusals of the library and
of its binding, which come before anything touches a GPU."""
import ctypes as C
import math

import numpy as np
import pytest

from oracle import i8


def test_quantize_by_hand():
    # largest 127: scale 1, halves to the even whole number
    q, s = i8.quantize(np.array([[127.0, 0.5, 1.5, -2.5, -0.5, 2.6]], np.float32))
    assert s[0] == 1 and q.tolist() == [[127, 0, 2, -2, 0, 3]]
    # largest 254: scale 2
    q, s = i8.quantize(np.array([[-254.0, 1.0, 3.0, 5.0, 253.0]], np.float32))
    assert s[0] == 2 and q.tolist() == [[-127, 0, 2, 2, 126]]
    q, s = i8.quantize(np.array([[1.0, 2.0, 4.0]], np.float32), np.array([127.0, 1.0, 0.125], np.float32))
    assert s[0] == 1 and q.tolist() == [[127, 2, 0]]


def test_quantize_special_rows():
    x = np.zeros((4, 3), np.float32)
    x[1, 0], x[2, 1], x[3, 2] = np.nan, np.inf, np.float32(2.0 ** -149)
    q, s = i8.quantize(x)
    assert not q.any() and s[0] == 0 and np.isnan(s[1]) and np.isnan(s[2]) and s[3] == 0


def test_product_by_hand():
    xq, xs = np.array([[2, -3]], np.int8), np.array([0.5], np.float32)
    wq, ws = np.array([[10, -128], [0, 127]], np.int8), np.array([2.0, 4.0], np.float32)
    # zeros 128: 20 + 384 = 404; -381
    assert i8.product(xq, xs, wq, ws).tolist() == [[404.0, -762.0]]
    # levels (10 + 128 - 0, 0) and (0 + 128 - 255, 127 - 127): 2 * 138, 2 * -127
    z = np.array([0, 255], np.uint8)
    assert i8.product(xq, xs, wq, ws, z, np.array([1.0, -1.0])).tolist() == [[277.0, -3 * 0 - 509.0]]


def test_route_by_hand():
    x = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    ids, w = i8.route(x, 2, renorm=False)
    assert ids.tolist() == [[2, 1]] and np.allclose(w, [[0.5, 0.25]])
    ids, w = i8.route(x, 3, renorm=True, scale=2.0)            # ties: the lower index
    assert ids.tolist() == [[2, 1, 0]] and np.allclose(w, [[8 / 7, 4 / 7, 2 / 7]])
    # the bias moves the choice, not the weight
    ids, w = i8.route(x, 1, bias=np.array([0.0, 0.0, 0.0, 1.0]), renorm=False)
    assert ids.tolist() == [[3]] and np.allclose(w, [[0.125]])
    # sigmoid: log 1 -> 1/2, log 4 -> 4/5; groups {0, 1} and {2, 3} by one or two of their best
    x = np.log(np.array([[3.0, 3.0, 4.0, 1.0]]))
    for best, want in ((1, 2), (2, 0)):
        ids, w = i8.route(x, 1, "sigmoid", None, 2, 1, best, renorm=False)
        assert ids.tolist() == [[want]] and np.allclose(w, [[0.8 if want == 2 else 0.75]])


def test_route_masked_rows():
    ninf = -math.inf
    ids, w = i8.route(np.array([[ninf, ninf, ninf], [ninf, 0.0, float("nan")]]), 2)
    assert ids.tolist() == [[0, 1], [1, 0]] and w.tolist() == [[0.0, 0.0], [1.0, 0.0]]


def test_moe_of_identity_experts():
    """One expert whose gate and up rows make h a known row, and a down matrix of one column."""
    x = np.array([[127.0, 64.0]], np.float32)
    gu = (np.array([[[1, 0], [0, 1]]], np.int8), np.array([[1.0, 1.0]], np.float32), None)
    dn = (np.array([[[1], [2]]], np.int8), np.array([[1.0, 0.5]], np.float32), None)
    y, _ = i8.moe(x, np.array([[0, 5]]), np.array([[0.5, 9.0]], np.float32), gu, dn, 1)
    h = 127.0 / (1 + math.exp(-127.0)) * 64.0      # its code is 127, its scale h / 127
    assert np.allclose(y, [[0.5 * h, 0.5 * h]])


# -------------------------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    import os
    from post_weight_quantization_05_amd import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.load()


A, ODD = C.c_void_p(4096), C.c_void_p(4097)


def test_pitch(lib):
    assert [lib.qz_i8_pitch(c) for c in (1, 128, 129, 65536, 0, -1, 65537)] == [128, 128, 256, 65536, -1, -1, -1]


def _refused(lib, fn, args, what, status=-1):
    assert getattr(lib, fn)(*args, None) == status
    assert what.encode() in lib.qz_last_error(), lib.qz_last_error()


@pytest.mark.parametrize("change,what", [
    ({1: 7}, "dtype"), ({2: -1}, "rows"), ({2: 2 ** 24 + 1}, "rows"), ({3: 0}, "cols"), ({3: 65537, 4: 70000}, "cols"),
    ({4: 15}, "ldx"), ({0: None}, "null"), ({6: None}, "null"), ({7: None}, "null"), ({6: C.c_void_p(4104)}, "16-byte"),
    ({0: ODD}, "aligned"), ({5: ODD}, "aligned"), ({7: ODD}, "aligned"), ({8: ODD}, "aligned"), ({9: ODD}, "aligned")])
def test_quantize_refusals(lib, change, what):
    a = [A, 0, 4, 16, 16, A, A, A, A, A]
    for i, v in change.items():
        a[i] = v
    _refused(lib, "qz_i8_quantize", a, what)


def test_quantize_and_packing_of_nothing(lib):
    assert lib.qz_i8_quantize(None, 0, 0, 16, 16, None, None, None, None, None, None) == 0
    assert lib.qz_i8_pack(None, 0, 16, None, None) == 0 and lib.qz_i8_unpack(None, 0, 16, None, None) == 0
    for fn in ("qz_i8_pack", "qz_i8_unpack"):
        _refused(lib, fn, [A, 4, 0, A], "cols")
        _refused(lib, fn, [A, -1, 16, A], "rows")
        _refused(lib, fn, [None, 4, 16, A], "null")
        _refused(lib, fn, [A, 4, 16, None], "null")
    _refused(lib, "qz_i8_pack", [A, 4, 16, C.c_void_p(4100)], "16-byte")
    _refused(lib, "qz_i8_unpack", [C.c_void_p(4100), 4, 16, A], "16-byte")


MATMUL = [A, A, A, 4, A, A, A, 8, 16, A, A, 0, 8, A, 1 << 40]
LINEAR = [A, 0, 4, 16, A, A, A, A, 8, 16, A, A, 0, 8, A, 1 << 40]


@pytest.mark.parametrize("fn,base,change,what", [
    ("qz_i8_matmul", MATMUL, {3: -1}, "need"), ("qz_i8_matmul", MATMUL, {3: 2 ** 20 + 1}, "need"),
    ("qz_i8_matmul", MATMUL, {7: 2 ** 24 + 1, 12: 2 ** 25}, "need"), ("qz_i8_matmul", MATMUL, {8: 65537}, "need"),
    ("qz_i8_matmul", MATMUL, {8: 0}, "need"), ("qz_i8_matmul", MATMUL, {11: 2}, "output dtype"),
    ("qz_i8_matmul", MATMUL, {12: 7}, "ldy"), ("qz_i8_matmul", MATMUL, {0: None}, "null"),
    ("qz_i8_matmul", MATMUL, {1: None}, "null"), ("qz_i8_matmul", MATMUL, {4: None}, "null"),
    ("qz_i8_matmul", MATMUL, {5: None}, "null"), ("qz_i8_matmul", MATMUL, {10: None}, "null"),
    ("qz_i8_matmul", MATMUL, {2: None}, "row sums"), ("qz_i8_matmul", MATMUL, {0: C.c_void_p(4104)}, "16-byte"),
    ("qz_i8_matmul", MATMUL, {4: C.c_void_p(4104)}, "16-byte"), ("qz_i8_matmul", MATMUL, {1: ODD}, "aligned"),
    ("qz_i8_matmul", MATMUL, {2: ODD}, "aligned"), ("qz_i8_matmul", MATMUL, {5: ODD}, "aligned"),
    ("qz_i8_matmul", MATMUL, {9: ODD}, "aligned"), ("qz_i8_matmul", MATMUL, {10: ODD}, "aligned"),
    ("qz_i8_linear", LINEAR, {1: 5}, "dtype"), ("qz_i8_linear", LINEAR, {3: 15}, "ldx"),
    ("qz_i8_linear", LINEAR, {2: -1}, "need"), ("qz_i8_linear", LINEAR, {9: 65537, 3: 70000}, "need"),
    ("qz_i8_linear", LINEAR, {0: None}, "null"), ("qz_i8_linear", LINEAR, {0: ODD}, "aligned"),
    ("qz_i8_linear", LINEAR, {4: ODD}, "aligned"), ("qz_i8_linear", LINEAR, {5: None}, "null"),
    ("qz_i8_linear", LINEAR, {12: 9}, "output dtype"), ("qz_i8_linear", LINEAR, {13: 7}, "ldy")])
def test_product_refusals(lib, fn, base, change, what):
    a = list(base)
    for i, v in change.items():
        a[i] = v
    _refused(lib, fn, a, what)


def test_products_of_nothing_and_workspaces(lib):
    a = list(MATMUL)
    a[3] = 0
    assert lib.qz_i8_matmul(*a, None) == 0
    a = list(LINEAR)
    a[8] = 0
    assert lib.qz_i8_linear(*a, None) == 0
    assert lib.qz_i8_linear_workspace(4, 8, 65537) == 0 and lib.qz_i8_matmul_workspace(-1, 8, 16) == 0
    for fn, base, query in (("qz_i8_linear", LINEAR, lib.qz_i8_linear_workspace),
                            ("qz_i8_matmul", MATMUL, lib.qz_i8_matmul_workspace)):
        for n, d_o, d_i in ((300, 8, 16), (300, 200, 4096), (5, 64, 20000)):
            need = query(n, d_o, d_i)
            if not need:
                continue
            a = list(base)
            if fn == "qz_i8_linear":
                a[2], a[3], a[8], a[9], a[13] = n, d_i, d_o, d_i, d_o
            else:
                a[3], a[7], a[8], a[12] = n, d_o, d_i, d_o
            a[-1] = need - 1
            _refused(lib, fn, a, "too small", -6)
            a[-2:] = None, need
            _refused(lib, fn, a, "too small", -6)
            a[-2:] = C.c_void_p(4096 + 128), need
            _refused(lib, fn, a, "256-byte", -6)


def _router(**kw):
    from post_weight_quantization_05_amd import _lib
    v = dict(struct_size=C.sizeof(_lib.QzRouter), n_experts=16, top_k=2, n_groups=4, top_groups=2, group_best=2,
             flags=3, scale=1.0)
    v.update(kw)
    return _lib.QzRouter(**v)


@pytest.mark.parametrize("params,what", [
    (dict(struct_size=4), "struct_size"), (dict(n_experts=0), "n_experts"), (dict(n_experts=513), "n_experts"),
    (dict(n_groups=0), "n_groups"), (dict(n_groups=3), "n_groups"), (dict(n_experts=130, n_groups=65), "n_groups"),
    (dict(top_groups=0), "top_groups"), (dict(top_groups=5), "top_groups"), (dict(group_best=0), "group_best"),
    (dict(group_best=3), "group_best"), (dict(top_k=0), "top_k"), (dict(top_k=9), "top_k"),
    (dict(n_experts=64, top_k=17), "top_k"), (dict(flags=4), "flags"), (dict(scale=float("nan")), "scale"),
    (dict(scale=float("inf")), "scale")])
def test_router_refusals(lib, params, what):
    _refused(lib, "qz_route", [A, 0, 4, 1000, C.byref(_router(**params)), A, A, A], what)


@pytest.mark.parametrize("change,what", [
    ({1: 3}, "dtype"), ({2: -1}, "need"), ({2: 2 ** 24 + 1}, "need"), ({3: 15}, "ldl"), ({0: None}, "null"),
    ({4: None}, "params"), ({6: None}, "null"), ({7: None}, "null"), ({0: ODD}, "aligned"), ({5: ODD}, "aligned"),
    ({6: ODD}, "aligned"), ({7: ODD}, "aligned")])
def test_route_refusals(lib, change, what):
    a = [A, 0, 4, 16, C.byref(_router()), A, A, A]
    for i, v in change.items():
        a[i] = v
    _refused(lib, "qz_route", a, what)
    a[0], a[1], a[2], a[3], a[4] = None, 0, 0, 16, C.byref(_router())
    assert lib.qz_route(*a, None) == 0


MOE = [A, 0, 4, 16, 16, 32, 8, 2, A, A, A, A, A, A, A, A, A, A, 1 << 40]


@pytest.mark.parametrize("change,what", [
    ({1: 2}, "dtype"), ({2: -1}, "need"), ({2: 2 ** 20 + 1}, "need"), ({3: 15}, "ldx"), ({4: 0}, "need"),
    ({4: 65537}, "need"), ({5: 0}, "need"), ({5: 65537}, "need"), ({3: 65536, 4: 65536, 5: 32768}, "f pitch"), ({6: 0}, "n_experts"), ({6: 513}, "n_experts"),
    ({7: 0}, "top_k"), ({7: 17}, "top_k"), ({2: 2 ** 20, 3: 4096, 4: 4096}, "in parts"), ({0: None}, "null"),
    ({8: None}, "null"), ({9: None}, "null"), ({10: None}, "null"), ({11: None}, "null"), ({13: None}, "null"),
    ({14: None}, "null"), ({16: None}, "null"), ({10: C.c_void_p(4104)}, "16-byte"), ({13: C.c_void_p(4104)}, "16-byte"),
    ({0: ODD}, "aligned"), ({8: ODD}, "aligned"), ({9: ODD}, "aligned"), ({11: ODD}, "aligned"), ({16: ODD}, "aligned")])
def test_moe_refusals(lib, change, what):
    a = list(MOE)
    for i, v in change.items():
        a[i] = v
    _refused(lib, "qz_i8_moe", a, what)


def test_moe_workspace(lib):
    need = lib.qz_i8_moe_workspace(4, 16, 32, 8, 2)
    assert need > 0 and lib.qz_i8_moe_workspace(4, 16, 32, 8, 17) == 0
    for ws, size, what in ((A, need - 1, "too small"), (None, need, "too small"), (C.c_void_p(4096 + 64), need, "256-byte")):
        a = list(MOE)
        a[-2:] = ws, size
        _refused(lib, "qz_i8_moe", a, what, -6)
    a = list(MOE)
    a[2] = 0
    assert lib.qz_i8_moe(*a, None) == 0


def test_binding_refuses_before_the_library():
    import torch
    import post_weight_quantization_05_amd as q
    x = torch.zeros((2, 16))
    for call in (lambda: q.qz_i8_quantize(x), lambda: q.qz_route(x, 2), lambda: q.qz_i8_pack(x.to(torch.uint8)),
                 lambda: q.qz_i8_unpack(x.to(torch.int8), 16),
                 lambda: q.qz_i8_linear(x, x.to(torch.int8), x[:, 0]),
                 lambda: q.qz_i8_matmul(x.to(torch.int8), x[:, 0], x.to(torch.int8), x[:, 0], 16)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for args in ((1, 64, 32, 2 ** 32 + 8, 2), (1, 64, 32, 8, 2 ** 32 + 2)):
        with pytest.raises(ValueError, match="32 bits"):
            q.qz_i8_moe_workspace(*args)
    assert q.qz_i8_moe_workspace(1, 64, 32, 8, 2) > 0
