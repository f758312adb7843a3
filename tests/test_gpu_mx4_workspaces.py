"""GPU: the MX4 operators in workspaces of the caller's, of exactly the size that the query gives, with
any bytes in them before the call and guards on both sides."""
import ctypes as C

import numpy as np
import pytest

from gpu_util import qz

pytestmark = pytest.mark.gpu


def _held(need, fill):
    """(workspace of `need` bytes, check that the bytes around it are as they were)."""
    import torch
    whole = torch.full((need + 1024,), fill, dtype=torch.uint8, device="cuda")
    at = 512 - whole.data_ptr() % 256
    ws = whole[at:at + need]
    assert ws.data_ptr() % 256 == 0 or need == 0

    def around():
        assert (whole[:at] == fill).all() and (whole[at + need:] == fill).all()
    return ws, around


def _stored(rows, cols, gen):
    import torch
    return qz().qz_mx4_quantize(torch.randn((rows, cols), device="cuda", generator=gen))


# n, d_i, d_o: few tokens, tiles with one split and with several, rows that are copied first
PRODUCTS = [(1, 64, 5), (3, 95, 45), (40, 1056, 130), (300, 512, 300), (262, 13184, 3687), (300, 12079, 231),
            (725, 9, 10891), (1, 1, 1), (1996, 3531, 2059)]


@pytest.mark.parametrize("n,d_i,d_o", PRODUCTS)
def test_products(n, d_i, d_o):
    import torch
    q = qz()
    gen = torch.Generator("cuda").manual_seed(n + d_i)
    codes, scales = _stored(d_o, d_i, gen)
    x = torch.randn((n, d_i), device="cuda", generator=gen).to(torch.bfloat16)
    xc, xs = q.qz_mx4_quantize(x)
    want = q.qz_mx4_linear(x, codes, scales)
    need = q.lib().qz_mx4_linear_workspace(x.data_ptr(), n, d_i, d_o, d_i)
    assert need <= q.qz_mx4_linear_workspace(n, d_o, d_i)
    for size in (need, q.qz_mx4_linear_workspace(n, d_o, d_i)):
        for fill in (0, 255):
            ws, around = _held(size, fill)
            assert torch.equal(q.qz_mx4_linear(x, codes, scales, ws=ws), want)
            around()
    if need:
        with pytest.raises(q.QzError, match="workspace"):
            q.qz_mx4_linear(x, codes, scales, ws=ws[:need - 1])
        with pytest.raises(q.QzError, match="aligned"):
            q.qz_mx4_linear(x, codes, scales, ws=torch.empty(need + 256, dtype=torch.uint8, device="cuda")[16:])
    want = q.qz_mx4_matmul(xc, xs, codes, scales, d_i)
    need = q.qz_mx4_matmul_workspace(n, d_o, d_i)
    for fill in (0, 255):
        ws, around = _held(need, fill)
        assert torch.equal(q.qz_mx4_matmul(xc, xs, codes, scales, d_i, ws=ws), want)
        around()
    if need:
        with pytest.raises(q.QzError, match="workspace"):
            q.qz_mx4_matmul(xc, xs, codes, scales, d_i, ws=ws[:need - 1])


# n, d, f, experts, top_k: one token, every expert chosen, several tiles of pairs, ragged rows
LAYERS = [(1, 64, 32, 4, 1), (1, 33, 1, 256, 16), (16, 100, 65, 128, 7), (17, 100, 65, 128, 7), (256, 70, 33, 5, 5),
          (48, 256, 96, 64, 6), (7, 2080, 544, 8, 2), (256, 64, 32, 256, 16)]


@pytest.mark.parametrize("n,d,f,E,k", LAYERS)
def test_expert_layer(n, d, f, E, k):
    import torch
    q = qz()
    gen = torch.Generator("cuda").manual_seed(n + d + f)
    x = torch.randn((n, d), device="cuda", generator=gen).to(torch.bfloat16)
    router = torch.randn((E, d), device="cuda", generator=gen) / np.sqrt(d)
    gu, gs = (a.view(E, 2 * f, -1) for a in _stored(E * 2 * f, d, gen))
    dn, ds = (a.view(E, d, -1) for a in _stored(E * d, f, gen))
    want = q.qz_mx4_moe(x, router, gu, gs, dn, ds, k, routing=True)
    need = q.qz_mx4_moe_workspace(n, d, f, E, k)
    for fill in (0, 255, 127):
        ws, around = _held(need, fill)
        got = q.qz_mx4_moe(x, router, gu, gs, dn, ds, k, routing=True, ws=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        around()
    with pytest.raises(q.QzError, match="workspace"):
        q.qz_mx4_moe(x, router, gu, gs, dn, ds, k, ws=ws[:need - 1])
    p = q._moe_params(E, k, True)
    assert q.lib().qz_mx4_moe_workspace(n, d, f, C.byref(p)) == need


def test_no_bytes_around_the_results():
    """Quantised codes, factors and values, unpacked integers: exactly their own bytes (odd sizes)."""
    import torch
    q = qz()
    L = q.lib()
    stream = torch.cuda.current_stream().cuda_stream
    for rows, cols in ((1, 1), (3, 31), (5, 33), (7, 200), (33, 1056), (1, 64)):
        blocks = -(-cols // 32)
        for dtype, code, size in ((torch.bfloat16, 0, 2), (torch.float32, 1, 4)):
            w = torch.randn((rows, cols), device="cuda").to(dtype)
            c, s, v = q.qz_mx4_quantize(w, rule="least", values=True)
            (hc, a1), (hs, a2), (hv, a3) = _held(rows * 16 * blocks, 7), _held(rows * blocks, 7), _held(rows * cols * size, 7)
            assert L.qz_mx4_quantize(w.data_ptr(), code, rows, cols, cols, 1, None, hc.data_ptr(), hs.data_ptr(),
                                     hv.data_ptr(), stream) == 0
            torch.cuda.synchronize()
            assert torch.equal(hc.view_as(c), c) and torch.equal(hs.view_as(s), s)
            assert torch.equal(hv.view(dtype).view_as(v), v)
            for a in (a1, a2, a3):
                a()
        i, f, z = q.qz_mx4_unpack(c, s, cols)
        (hi, a1), (hf, a2), (hz, a3) = _held(4 * rows * cols, 7), _held(4 * rows * blocks, 7), _held(rows * blocks, 7)
        assert L.qz_mx4_unpack(c.data_ptr(), s.data_ptr(), rows, cols, hi.data_ptr(), hf.data_ptr(), hz.data_ptr(),
                               stream) == 0
        torch.cuda.synchronize()
        assert torch.equal(hi.view(torch.int32).view_as(i), i) and torch.equal(hf.view(torch.float32).view_as(f), f)
        assert torch.equal(hz.view_as(z), z)
        for a in (a1, a2, a3):
            a()
