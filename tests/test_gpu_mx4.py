"""GPU: the microscaled 4-bit operators against the oracle's definitions in 64 bits.

Quantisation is compared bit for bit.  Products are compared exactly where every partial sum
is a small multiple of a power of two (then fp32 sums have no rounding, whatever their order),
and within a derived bound on ordinary values:

  fp32 sums: the matrix cores add 32 (bf16) or 128 (MX4) products into one accumulator at a
  time, so a sum of K products passes through at most K / 32 roundings of the accumulator, 32
  inside a step, and the joins of the wavefronts' partial sums (below 32); each rounding is at
  most 2^-23 (truncation) of a partial sum, and those are at most S = sum |x w|:
      |error| <= (K / 32 + 64) 2^-23 S,
  plus half a step of the output type, 2^-8 |y| in bf16 and 2^-24 |y| in fp32."""
import numpy as np
import pytest

from gpu_util import qz, to_dev, to_host
from oracle import mx4, objective

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _t():
    import torch
    return torch


def _dtype(name):
    return {"bf16": _t().bfloat16, "f32": _t().float32}[name]


def _bf16(a):
    """Values rounded to bf16, as float64, and the device tensor."""
    t = _t().from_numpy(np.ascontiguousarray(a, np.float32)).to(_t().bfloat16)
    return t.double().numpy(), t.cuda()


def _host(t):
    return t.double().cpu().numpy() if t.is_floating_point() else to_host(t)


def _random_codes(rng, rows, cols, e_lo=126, e_hi=129):
    """Codes (zero past cols) and factors."""
    g = -(-cols // 32)
    c = rng.integers(0, 16, (rows, 32 * g)).astype(np.uint8)
    c[:, cols:] = 0
    return c[:, 0::2] | (c[:, 1::2] << 4), rng.integers(e_lo, e_hi, (rows, g)).astype(np.uint8)


def _sum_bound(K, S, out, y):
    return (K / 32 + 64) * 2.0 ** -23 * S + HALF[out] * np.abs(y)


# ------------------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (2, 32), (5, 33), (70, 200), (33, 1056),
                                       (64, 4096), (300, 520), (1, 25600)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rule,weighted", [("floor", False), ("least", False), ("least", True)])
def test_quantize_bit_exact(rows, cols, dtype, rule, weighted):
    q = qz()
    rng = np.random.default_rng([rows, cols])
    w = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)))
    w[rng.random((rows, cols)) < 0.1] = 0.0
    near = rng.random((rows, cols)) < 0.3     # many values on the grid, on ties and at 6 .. 8
    w = np.where(near, np.round(w * 8) / 8 * 2, w)
    x = _t().from_numpy(w.astype(np.float32)).to(_dtype(dtype))
    h = np.exp(rng.standard_normal(cols)).astype(np.float32) if weighted else None
    c, s, v = q.qz_mx4_quantize(x.cuda(), rule=rule, colw=None if h is None else to_dev(h), values=True)
    c_ref, s_ref = mx4.quantize(x.float().numpy(), rule, h)
    np.testing.assert_array_equal(to_host(s), s_ref)
    np.testing.assert_array_equal(to_host(c), c_ref)
    assert v.dtype == x.dtype
    np.testing.assert_array_equal(_host(v), mx4.values(c_ref, s_ref, cols))
    c2, s2 = q.qz_mx4_quantize(x.cuda(), rule=rule, colw=None if h is None else to_dev(h))
    assert _t().equal(c, c2) and _t().equal(s, s2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rule", ["floor", "least"])
def test_quantize_special_values(dtype, rule):
    q = qz()
    top = float(_t().finfo(_dtype(dtype)).max)
    rows = [[0.0] * 40, [-0.0] * 40, [2.0 ** -126] * 40, [2.0 ** -130, -(2.0 ** -128)] * 20,
            [2.0 ** -133] + [0.0] * 39, [top, -top] * 20, [1.0] * 32 + [float("nan")] + [2.0] * 7,
            [float("inf")] + [1.0] * 39, [-float("inf"), float("nan")] * 20, [1e-30, 1e30] * 20,
            [7.0, 0.5, -3.0, -0.0] * 10, [5.0, -5.0, 2.5, 1.75, 0.75, 0.25, 3.5, 1.25] * 5]
    x = _t().tensor(rows, dtype=_t().float32).to(_dtype(dtype))
    c, s, v = q.qz_mx4_quantize(x.cuda(), rule=rule, values=True)
    c_ref, s_ref = mx4.quantize(x.float().numpy(), rule)
    np.testing.assert_array_equal(to_host(s), s_ref)
    np.testing.assert_array_equal(to_host(c), c_ref)
    np.testing.assert_array_equal(_host(v), mx4.values(c_ref, s_ref, 40))


def test_quantize_strided_and_unaligned_rows():
    q, torch = qz(), _t()
    base = torch.randn((37, 300), device="cuda")
    for x in (base[:, 5:205], base[:, 4:132], base[::2, 1:97], base[3:4, 7:39],
              base.to(torch.bfloat16)[:, 3:131], base.to(torch.bfloat16)[:, 8:200]):
        c, s, v = q.qz_mx4_quantize(x, rule="least", values=True)
        c_ref, s_ref = mx4.quantize(x.float().cpu().numpy(), "least")
        np.testing.assert_array_equal(to_host(c), c_ref)
        np.testing.assert_array_equal(to_host(s), s_ref)
        np.testing.assert_array_equal(_host(v), mx4.values(c_ref, s_ref, x.shape[1]))


@pytest.mark.parametrize("cols", [32, 33, 96])
def test_unpack(cols):
    q = qz()
    rng = np.random.default_rng(cols)
    codes, scales = _random_codes(rng, 17, cols, 0, 256)
    scales[0, 0], scales[1, 0], scales[2, 0], scales[3, 0] = 0, 1, 2, 255
    c, s, z = q.qz_mx4_unpack(to_dev(codes), to_dev(scales), cols)
    np.testing.assert_array_equal(to_host(c), 2 * mx4.elements(codes, cols))
    want = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 128))
    np.testing.assert_array_equal(_host(s), want)
    assert not to_host(z).any()


# ---------------------------------------------------------------------------------- products
NS = [1, 2, 5, 15, 16, 17, 31, 33, 64, 65, 128, 129, 200, 257, 300]
SHAPES = [(32, 16), (1, 1), (31, 7), (33, 15), (64, 17), (96, 100), (200, 33), (512, 64),
          (640, 130), (1024, 257), (1056, 40), (2080, 520)]


def _cases():
    """Every n with some shape and every shape with some n, and the corners of both."""
    out = [(n, *SHAPES[i % len(SHAPES)]) for i, n in enumerate(NS)]
    out += [(NS[(5 * i + 3) % len(NS)], *s) for i, s in enumerate(SHAPES)]
    return sorted(set(out + [(300, 2080, 520), (1, 2080, 520), (257, 1, 1), (130, 96, 1030)]))


@pytest.mark.parametrize("n,d_i,d_o", _cases())
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_linear_exact(n, d_i, d_o, out):
    """Integers -8 .. 8 times multiples of 1/4 up to 12 (factors 1/2 .. 2): sums are multiples
    of 1/4 below 2^18, exact in fp32; bf16 output is the one rounding of that."""
    q = qz()
    rng = np.random.default_rng([n, d_i, d_o])
    x = rng.integers(-8, 9, (n, d_i)).astype(np.float64)
    codes, scales = _random_codes(rng, d_o, d_i)
    bias = rng.integers(-50, 50, d_o).astype(np.float32) if (n + d_o) % 2 else None
    y = x @ mx4.values(codes, scales, d_i).T + (0 if bias is None else bias)
    got = q.qz_mx4_linear(_bf16(x)[1], to_dev(codes), to_dev(scales),
                          bias=None if bias is None else to_dev(bias), out_dtype=_dtype(out))
    assert got.dtype == _dtype(out)
    want = _t().from_numpy(y).float().to(_dtype(out)).double().numpy()
    np.testing.assert_array_equal(_host(got), want)


@pytest.mark.parametrize("n,d_i,d_o", _cases())
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_matmul_exact(n, d_i, d_o, out):
    """Both factors 1/2 .. 2: products are multiples of 1/16 up to 144, sums below 2^19."""
    q = qz()
    rng = np.random.default_rng([n, d_i, d_o, 4])
    xc, xs = _random_codes(rng, n, d_i)
    codes, scales = _random_codes(rng, d_o, d_i)
    bias = rng.integers(-50, 50, d_o).astype(np.float32) if (n + d_o) % 2 else None
    y = mx4.values(xc, xs, d_i) @ mx4.values(codes, scales, d_i).T + (0 if bias is None else bias)
    got = q.qz_mx4_matmul(to_dev(xc), to_dev(xs), to_dev(codes), to_dev(scales), d_i,
                          bias=None if bias is None else to_dev(bias), out_dtype=_dtype(out))
    want = _t().from_numpy(y).float().to(_dtype(out)).double().numpy()
    np.testing.assert_array_equal(_host(got), want)


@pytest.mark.parametrize("n,d_i,d_o", [(1, 4096, 512), (13, 5120, 300), (100, 1408, 256), (515, 2048, 384)])
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_products_of_ordinary_values(n, d_i, d_o, four, out):
    q = qz()
    rng = np.random.default_rng([n, d_i])
    x, xd = _bf16(rng.standard_t(4, (n, d_i)))
    w = (rng.standard_normal((d_o, d_i)) * 0.015).astype(np.float32)
    codes, scales = mx4.quantize(w)
    wv = mx4.values(codes, scales, d_i)
    if four:
        xc, xs = q.qz_mx4_quantize(xd)
        got = q.qz_mx4_matmul(xc, xs, to_dev(codes), to_dev(scales), d_i, out_dtype=_dtype(out))
        x = mx4.values(*mx4.quantize(x), d_i)
    else:
        got = q.qz_mx4_linear(xd, to_dev(codes), to_dev(scales), out_dtype=_dtype(out))
    y = x @ wv.T
    assert (np.abs(_host(got) - y) <= _sum_bound(d_i, np.abs(x) @ np.abs(wv).T, out, y)).all()


def test_far_factors():
    """The ends of the factor's range: 2^-127 (subnormal weights) against 2^100 inputs, and
    products that cancel exactly."""
    q = qz()
    rng = np.random.default_rng(5)
    codes, _ = _random_codes(rng, 40, 96)
    scales = np.zeros((40, 3), np.uint8)
    scales[20:] = 1
    x, xd = _bf16(np.ldexp(rng.integers(-8, 9, (20, 96)).astype(np.float64), 100))
    want = x @ mx4.values(codes, scales, 96).T
    got = q.qz_mx4_linear(xd, to_dev(codes), to_dev(scales), out_dtype=_t().float32)
    np.testing.assert_array_equal(_host(got), want)
    xc, _ = _random_codes(rng, 20, 96)
    xs = np.full((20, 3), 227, np.uint8)
    want = mx4.values(xc, xs, 96) @ mx4.values(codes, scales, 96).T
    got = q.qz_mx4_matmul(to_dev(xc), to_dev(xs), to_dev(codes), to_dev(scales), 96, out_dtype=_t().float32)
    np.testing.assert_array_equal(_host(got), want)


@pytest.mark.parametrize("n", [1, 16, 40, 130, 300])
@pytest.mark.parametrize("d_i", [256, 1056])
def test_nan_stays_in_its_row(n, d_i):
    q, torch = qz(), _t()
    rng = np.random.default_rng(n)
    x = rng.integers(-8, 9, (n, d_i)).astype(np.float64)
    codes, scales = _random_codes(rng, 70, d_i)
    scales[33, -1] = 255
    bad = n // 2
    x[bad, 3] = np.nan
    got = _host(q.qz_mx4_linear(_bf16(x)[1], to_dev(codes), to_dev(scales), out_dtype=torch.float32))
    assert np.isnan(got[bad]).all() and np.isnan(got[:, 33]).all()
    keep_t, keep_r = np.arange(n) != bad, np.arange(70) != 33
    want = x[keep_t] @ mx4.values(codes, scales, d_i)[keep_r].T
    np.testing.assert_array_equal(got[keep_t][:, keep_r], want)
    xc, xs = _random_codes(rng, n, d_i)
    xs[bad, 0] = 255
    got = _host(q.qz_mx4_matmul(to_dev(xc), to_dev(xs), to_dev(codes), to_dev(scales), d_i,
                                out_dtype=torch.float32))
    assert np.isnan(got[bad]).all() and np.isnan(got[:, 33]).all()
    want = mx4.values(xc, xs, d_i)[keep_t] @ mx4.values(codes, scales, d_i)[keep_r].T
    np.testing.assert_array_equal(got[keep_t][:, keep_r], want)


@pytest.mark.parametrize("n,d_i,d_o", [(1, 128, 50), (16, 200, 33), (70, 96, 129), (300, 512, 300)])
def test_strided_inputs_and_outputs(n, d_i, d_o):
    """Rows inside wider buffers, at odd offsets: nothing between the rows is touched."""
    q, torch = qz(), _t()
    rng = np.random.default_rng([n, d_o])
    x = rng.integers(-8, 9, (n, d_i)).astype(np.float64)
    codes, scales = _random_codes(rng, d_o, d_i)
    want = x @ mx4.values(codes, scales, d_i).T
    xc, xs = _random_codes(rng, n, d_i)
    want4 = mx4.values(xc, xs, d_i) @ mx4.values(codes, scales, d_i).T
    for off, dtype in ((0, torch.float32), (1, torch.bfloat16), (8, torch.bfloat16), (3, torch.float32)):
        wide = torch.full((n, d_i + 19), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, off:off + d_i] = _bf16(x)[1]
        for four in (False, True):
            y = torch.full((n + 2, d_o + 11), 7.0, dtype=dtype, device="cuda")
            part = y[1:n + 1, off:off + d_o]
            if four:
                q.qz_mx4_matmul(to_dev(xc), to_dev(xs), to_dev(codes), to_dev(scales), d_i, out=part)
            else:
                q.qz_mx4_linear(wide[:, off:off + d_i], to_dev(codes), to_dev(scales), out=part)
            ref = torch.full_like(y, 7.0)
            ref[1:n + 1, off:off + d_o] = torch.from_numpy(want4 if four else want).to(dtype).cuda()
            assert torch.equal(y, ref), (off, dtype, four)


# Sizes that reach each kernel shape of the products, unsplit and split along d_i: (n, d_i, d_o).
EACH_LINEAR = [
    (3, 95, 45), (2, 1179, 33), (16, 2080, 97), (1, 64, 9737), (13, 200, 9741), (17, 15, 4231), (21, 352, 4117),
    (582, 475, 1365), (75, 1056, 2049), (18, 9, 9839), (25, 96, 8517), (17, 12123, 2833), (231, 27, 8457),
    (747, 9209, 351), (66, 35, 10915), (300, 12079, 231), (1547, 21, 4875), (1615, 8991, 359), (514, 15, 7289),
    (34, 19, 4289), (185, 11509, 803), (95, 10327, 2773), (328, 12069, 901), (725, 9, 10891), (1074, 3343, 3985), (1996, 3531, 2059)]
EACH_MATMUL = [
    (3, 95, 45), (2, 1179, 33), (16, 2080, 97), (325, 305, 1763), (217, 9, 2077), (171, 96, 2635), (52, 9, 8251),
    (49, 29, 8525), (618, 9719, 423), (154, 13, 11019), (522, 12065, 587), (194, 13, 9753), (678, 11513, 1693), (1343, 11213, 1799),
    (688, 645, 1089), (720, 10461, 359), (647, 19, 6225), (1487, 283, 10851), (833, 7663, 2307), (1651, 15, 2519), (1098, 9, 7213), (849, 9907, 3141)]


def _each(sizes, seed, matmul, integer):
    """(result, 64-bit result) of integers against random codes, computed on the GPU; integer: the
    values are multiples of `integer` and sums of their magnitudes stay below 2^24 of it."""
    q, torch = qz(), _t()
    n, d_i, d_o = sizes
    rng = np.random.default_rng([n, d_i, d_o, seed])
    codes, scales = _random_codes(rng, d_o, d_i)
    w = to_dev(mx4.values(codes, scales, d_i))
    bias = rng.integers(-50, 50, d_o).astype(np.float32) if (n + d_o) % 2 else None
    b = None if bias is None else to_dev(bias)
    if matmul:
        xc, xs = _random_codes(rng, n, d_i)
        x = to_dev(mx4.values(xc, xs, d_i))
        got = q.qz_mx4_matmul(to_dev(xc), to_dev(xs), to_dev(codes), to_dev(scales), d_i, bias=b,
                              out_dtype=torch.float32)
    else:
        xv, xd = _bf16(rng.integers(-8, 9, (n, d_i)))
        x = to_dev(xv)
        got = q.qz_mx4_linear(xd, to_dev(codes), to_dev(scales), bias=b, out_dtype=torch.float32)
    assert float((x.abs() @ w.abs().T).max()) + 50 < integer * 2.0 ** 24
    return got.double(), x @ w.T + (0 if b is None else b.double())


@pytest.mark.parametrize("sizes", EACH_LINEAR)
def test_linear_in_every_shape(sizes):
    got, want = _each(sizes, 0, False, 2.0 ** -2)
    assert _t().equal(got, want)


@pytest.mark.parametrize("sizes", EACH_MATMUL)
def test_matmul_in_every_shape(sizes):
    got, want = _each(sizes, 1, True, 2.0 ** -4)
    assert _t().equal(got, want)


@pytest.mark.parametrize("n", [1, 13, 40, 200, 700])
@pytest.mark.parametrize("d_i", [96, 544, 1056, 2080])
def test_factors_and_codes_at_any_address(n, d_i):
    """Factors at odd addresses, codes at an odd multiple of 16 bytes, as in one packed file."""
    q, torch = qz(), _t()
    rng = np.random.default_rng([n, d_i])

    def moved(a, off):
        buf = torch.full((a.size + off,), 255, dtype=torch.uint8, device="cuda")
        buf[off:] = to_dev(a).reshape(-1)
        return buf[off:].view(a.shape)

    codes, scales = _random_codes(rng, 77, d_i)
    x, xd = _bf16(rng.integers(-8, 9, (n, d_i)))
    xc, xs = _random_codes(rng, n, d_i)
    for off in (1, 2, 3):
        got = q.qz_mx4_linear(xd, moved(codes, 16 * off), moved(scales, off), out_dtype=torch.float32)
        np.testing.assert_array_equal(_host(got), x @ mx4.values(codes, scales, d_i).T)
        got = q.qz_mx4_matmul(moved(xc, 16), moved(xs, 4 - off), moved(codes, 16 * off), moved(scales, off),
                              d_i, out_dtype=torch.float32)
        np.testing.assert_array_equal(_host(got), mx4.values(xc, xs, d_i) @ mx4.values(codes, scales, d_i).T)


def test_products_past_32_bits():
    """Codes, inputs and outputs whose last bytes lie more than 2^32 bytes from their first."""
    q, torch = qz(), _t()
    d_o, d_i = 600_000, 16384
    g = torch.Generator("cuda").manual_seed(1)
    codes = torch.randint(0, 256, (d_o, d_i // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(126, 129, (d_o, d_i // 32), dtype=torch.uint8, device="cuda", generator=g)
    pick = torch.tensor([0, 1, 262143, 262144, 524287, 524288, d_o - 2, d_o - 1], device="cuda")
    w = mx4.values(to_host(codes[pick]), to_host(scales[pick]), d_i)
    for n in (1, 9, 300):
        x = torch.randint(-3, 4, (n, d_i), device="cuda", generator=g).to(torch.bfloat16)
        y = q.qz_mx4_linear(x, codes, scales, out_dtype=torch.float32)[:, pick]
        np.testing.assert_array_equal(_host(y), _host(x.double()) @ w.T)
        xc, xs = q.qz_mx4_quantize(x)     # -3 .. 3: exact in E2M1
        y = q.qz_mx4_matmul(xc, xs, codes, scales, d_i, out_dtype=torch.float32)[:, pick]
        np.testing.assert_array_equal(_host(y), _host(x.double()) @ w.T)
    del codes, scales, y
    wide = torch.zeros((1100, 1 << 21), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((1100, 1 << 21), dtype=torch.bfloat16, device="cuda")
    wide[:, :64] = torch.randint(-3, 4, (1100, 64), device="cuda", generator=g).to(torch.bfloat16)
    c, s = _random_codes(np.random.default_rng(2), 48, 64)
    q.qz_mx4_linear(wide[:, :64], to_dev(c), to_dev(s), out=out[:, 5:53])
    want = torch.from_numpy(_host(wide[:, :64].double()) @ mx4.values(c, s, 64).T).to(torch.bfloat16)
    assert torch.equal(out[:, 5:53].cpu(), want)
    assert not out[:, :5].any() and not out[:, 53:101].any()


def test_quantize_past_32_bits():
    q, torch = qz(), _t()
    rows, cols = 330_000, 8200
    w = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    w.normal_(generator=torch.Generator("cuda").manual_seed(4))
    pick = torch.tensor([0, 1, 131071, 131072, 261887, 261888, 261889, rows - 1], device="cuda")
    for rule in ("floor", "least"):
        c, s, v = q.qz_mx4_quantize(w, rule=rule, values=True)
        c_ref, s_ref = mx4.quantize(w[pick].float().cpu().numpy(), rule)
        np.testing.assert_array_equal(to_host(c[pick]), c_ref)
        np.testing.assert_array_equal(to_host(s[pick]), s_ref)
        np.testing.assert_array_equal(_host(v[pick].double()), mx4.values(c_ref, s_ref, cols))


def test_most_tokens():
    """2^20 tokens, the most that a call takes, through few and through ordinary rows of W."""
    q, torch = qz(), _t()
    g = torch.Generator("cuda").manual_seed(6)
    for d_i, d_o in ((2000, 5), (1024, 16), (320, 100)):
        codes, scales = _random_codes(np.random.default_rng(d_i), d_o, d_i)
        w = mx4.values(codes, scales, d_i)
        x = torch.randint(-3, 4, (1 << 20, d_i), device="cuda", generator=g).to(torch.bfloat16)
        pick = torch.tensor([0, 1, 65535, 524288, (1 << 20) - 17, (1 << 20) - 2, (1 << 20) - 1], device="cuda")
        want = _host(x[pick].double()) @ w.T
        y = q.qz_mx4_linear(x, to_dev(codes), to_dev(scales), out_dtype=torch.float32)
        np.testing.assert_array_equal(_host(y[pick]), want)
        xc, xs = q.qz_mx4_quantize(x)
        y = q.qz_mx4_matmul(xc, xs, to_dev(codes), to_dev(scales), d_i, out_dtype=torch.float32)
        np.testing.assert_array_equal(_host(y[pick]), want)


@pytest.mark.parametrize("n,d_i,d_o", [(1, 32, 1 << 24), (33, 20, 1 << 24), (1, 1 << 20, 40), (17, 1 << 20, 9),
                                       (100, (1 << 20) - 3, 70), (300, 1 << 20, 33)])
def test_most_rows_and_columns(n, d_i, d_o):
    """The largest d_o and d_i.  Inputs -1 .. 1, factors 1/2 .. 2: sums of magnitudes below 2^24
    quarters for 2^20 columns only on average, so bounds there and equality for the short rows."""
    q, torch = qz(), _t()
    rng = np.random.default_rng([n, d_i])
    codes, scales = _random_codes(rng, d_o, d_i)
    pick = np.unique(np.r_[:8, d_o // 2, d_o - 8:d_o])
    w = mx4.values(codes[pick], scales[pick], d_i)
    x, xd = _bf16(rng.integers(-1, 2, (n, d_i)))
    want, total = x @ w.T, np.abs(x) @ np.abs(w).T
    xc, xs = q.qz_mx4_quantize(xd)
    for y in (q.qz_mx4_linear(xd, to_dev(codes), to_dev(scales), out_dtype=torch.float32),
              q.qz_mx4_matmul(xc, xs, to_dev(codes), to_dev(scales), d_i, out_dtype=torch.float32)):
        got = _host(y[:, torch.from_numpy(pick).cuda()])
        if d_i <= 32:
            np.testing.assert_array_equal(got, want)
        else:
            assert (np.abs(got - want) <= _sum_bound(d_i, total, "f32", want)).all()


def test_quantize_past_2_32_pieces():
    """More than 2^32 pieces of eight columns: the index is 64 bits wide."""
    q, torch = qz(), _t()
    rows, cols = 4_200_000, 8192
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GB of free GPU memory")
    w = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    pick = torch.tensor([0, 1, 2097151, 2097152, 4194303, 4194304, rows - 1], device="cuda")
    w[pick] = torch.randn((7, cols), device="cuda").to(torch.bfloat16)
    c, s = q.qz_mx4_quantize(w)
    c_ref, s_ref = mx4.quantize(w[pick].float().cpu().numpy())
    np.testing.assert_array_equal(to_host(c[pick]), c_ref)
    np.testing.assert_array_equal(to_host(s[pick]), s_ref)
    others = torch.tensor([2, 2097150, 2097153, 4194302, 4194305, rows - 2], device="cuda")
    assert not c[others].any() and not s[others].any()


def test_empty_products():
    q, torch = qz(), _t()
    codes, scales = _random_codes(np.random.default_rng(0), 8, 64)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert q.qz_mx4_linear(x, to_dev(codes), to_dev(scales)).shape == (0, 8)
    c, s = q.qz_mx4_quantize(x)
    assert c.shape == (0, 32) and q.qz_mx4_matmul(c, s, to_dev(codes), to_dev(scales), 64).shape == (0, 8)
    x = torch.ones((3, 64), dtype=torch.bfloat16, device="cuda")
    assert q.qz_mx4_linear(x, to_dev(codes)[:0], to_dev(scales)[:0]).shape == (3, 0)


# --------------------------------------------------------------------------- the expert layer
def _moe_bound(x, router, gu, dn, k, renorm):
    """(y, |error| allowed).  Per pair: dg, du from the fp32 sums; |silu'| <= 1.1; the exponential,
    quotient and product of h: 16 steps of 2^-24; the split of h: 2^-16; the weight: 2^-20; then
    the down sum (value and remainder: twice the products) and the join of the experts."""
    f, d = gu.shape[1] // 2, x.shape[1]
    ids, p = mx4.route(x, router, k, renorm)
    y, err = np.zeros((len(x), dn.shape[1])), np.zeros((len(x), dn.shape[1]))
    eps_d, eps_f = (d / 32 + 64) * 2.0 ** -23, (2 * f / 32 + 64 + 32) * 2.0 ** -23
    for t in range(len(x)):
        for r, e in enumerate(ids[t]):
            a = gu[e] @ x[t]
            da = eps_d * (np.abs(gu[e]) @ np.abs(x[t]))
            g, u = a[:f], a[f:]
            s = g / (1 + np.exp(-g))
            h = s * u
            dh = 1.1 * da[:f] * (np.abs(u) + da[f:]) + np.abs(s) * da[f:] + np.abs(h) * (2.0 ** -20 + 2.0 ** -16)
            y[t] += p[t, r] * (dn[e] @ h)
            err[t] += p[t, r] * (np.abs(dn[e]) @ (dh + (eps_f + 2.0 ** -20) * np.abs(h)))
    return y, ids, p, err + 2.0 ** -8 * np.abs(y)


MOE = [  # n, d, f, experts, top_k, renorm, router type
    (1, 64, 32, 4, 1, True, "bf16"), (1, 256, 96, 8, 2, False, "bf16"), (3, 100, 33, 5, 5, True, "f32"),
    (7, 512, 128, 16, 4, True, "bf16"), (16, 128, 64, 128, 8, True, "bf16"), (17, 33, 1, 3, 2, False, "f32"),
    (40, 256, 160, 64, 6, False, "bf16"), (64, 96, 64, 4, 3, True, "f32"), (65, 64, 40, 256, 16, True, "bf16"),
    (130, 64, 32, 2, 1, False, "bf16"), (1, 1, 1, 1, 1, True, "f32"), (5, 1056, 544, 7, 2, True, "bf16")]


def _moe_inputs(case):
    n, d, f, E, k, renorm, rt = case
    rng = np.random.default_rng([n, d, f, E])
    x, xd = _bf16(rng.standard_normal((n, d)))
    router = (rng.standard_normal((E, d)) / np.sqrt(d)).astype(np.float32)
    rd = _t().from_numpy(router).to(_dtype(rt))
    gu = mx4.quantize(rng.standard_normal((E * 2 * f, d)).astype(np.float32) / np.sqrt(d))
    dn = mx4.quantize(rng.standard_normal((E * d, f)).astype(np.float32) / np.sqrt(f))
    stored = [a.reshape(E, b, -1) for a, b in zip((*gu, *dn), (2 * f, 2 * f, d, d))]
    return x, xd, rd.double().numpy(), rd.cuda(), stored, [to_dev(a) for a in stored]


@pytest.mark.parametrize("case", MOE)
def test_moe(case):
    q = qz()
    n, d, f, E, k, renorm, _ = case
    x, xd, router, rd, st, dev = _moe_inputs(case)
    want, ids, p, bound = _moe_bound(x, router, mx4.values(st[0], st[1], d), mx4.values(st[2], st[3], f), k, renorm)
    y, got_ids, w = q.qz_mx4_moe(xd, rd, *dev, k, renorm=renorm, routing=True)
    np.testing.assert_array_equal(to_host(got_ids), ids)
    # exp of a rounded difference below 2^5, the sum and the quotient: 2^-20 in all
    assert (np.abs(_host(w) - p) <= 2.0 ** -20 * p).all()
    assert (np.abs(_host(y) - want) <= bound).all(), np.max(np.abs(_host(y) - want) / bound)
    assert _t().equal(y, q.qz_mx4_moe(xd, rd, *dev, k, renorm=renorm))     # and again, to the bit


MOE_CROWDED = [  # experts that get many tokens: several tiles of pairs, the last one part full
    (256, 64, 40, 2, 1, True, "bf16"), (256, 96, 33, 3, 3, False, "f32"), (100, 256, 96, 1, 1, True, "bf16"),
    (33, 544, 300, 5, 4, True, "bf16"), (256, 33, 65, 256, 2, False, "bf16"), (16, 64, 96, 256, 15, True, "f32"),
    (15, 64, 96, 256, 16, True, "bf16"), (2, 2080, 1100, 12, 6, True, "bf16"), (48, 160, 520, 17, 16, False, "bf16"),
    (200, 2080, 40, 3, 3, True, "bf16"), (16, 2050, 40, 140, 3, False, "bf16"), (40, 2112, 33, 130, 5, True, "f32"),
    (256, 2056, 16, 256, 16, False, "f32"), (20, 4100, 300, 33, 4, True, "bf16")]


@pytest.mark.parametrize("case", MOE_CROWDED)
def test_moe_crowded(case):
    test_moe(case)


@pytest.mark.parametrize("case", [(2, 64, 1 << 20, 1, 1, True, "bf16"), (3, 1 << 20, 32, 1, 1, False, "f32")])
def test_moe_longest_rows(case):
    test_moe(case)


def test_moe_all_tokens_to_one_expert():
    """Every token takes the same two experts of many; the others' slots stay empty."""
    q, torch = qz(), _t()
    n, d, f, E, k = 70, 128, 48, 40, 2
    x, xd, router, rd, st, dev = _moe_inputs((n, d, f, E, k, True, "f32"))
    xd = xd.abs()
    rd[:] = 0
    rd[39], rd[7] = 2.0, 1.0
    x, router = _host(xd), _host(rd)
    want, ids, p, bound = _moe_bound(x, router, mx4.values(st[0], st[1], d), mx4.values(st[2], st[3], f), k, True)
    y, got, w = q.qz_mx4_moe(xd, rd, *dev, k, routing=True)
    assert (to_host(got) == [39, 7]).all() and (ids == [39, 7]).all()
    assert (np.abs(_host(y) - want) <= bound).all()


def test_moe_past_32_bits():
    """Experts whose weights begin more than 2^32 bytes from the first one's."""
    q, torch = qz(), _t()
    E, d, f = 256, 4096, 4160
    g = torch.Generator("cuda").manual_seed(3)
    gu = torch.randint(0, 256, (E, 2 * f, d // 2), dtype=torch.uint8, device="cuda", generator=g)
    dn = torch.randint(0, 256, (E, d, f // 2), dtype=torch.uint8, device="cuda", generator=g)
    gs = torch.full((E, 2 * f, d // 32), 118, dtype=torch.uint8, device="cuda")
    ds = torch.full((E, d, f // 32), 118, dtype=torch.uint8, device="cuda")
    x = torch.randn((2, d), device="cuda", generator=g).to(torch.bfloat16)
    router = torch.zeros((E, d), device="cuda")
    router[255], router[0], router[250] = x[0].float(), x[1].float(), x.float().sum(0) / 2
    xh, ids = _host(x), [255, 250, 0]
    # the same layer with those three experts alone
    parts = [to_host(a[ids]) for a in (gu, gs, dn, ds)]
    guv, dnv = mx4.values(parts[0], parts[1], d), mx4.values(parts[2], parts[3], f)
    want, sub, p, bound = _moe_bound(xh, _host(router[ids]), guv, dnv, 2, True)
    y, got, w = q.qz_mx4_moe(x, router, gu, gs, dn, ds, 2, routing=True)
    np.testing.assert_array_equal(to_host(got), np.array(ids)[sub])
    assert (np.abs(_host(y) - want) <= bound).all()


def test_moe_without_renorm_and_a_nan_router_row():
    """A NaN logit counts as -inf in the softmax over all experts too."""
    q, torch = qz(), _t()
    x, xd, router, rd, st, dev = _moe_inputs((6, 64, 32, 8, 2, False, "bf16"))
    r2 = rd.clone()
    r2[3] = float("nan")
    y, ids, w = q.qz_mx4_moe(xd, r2, *dev, 2, renorm=False, routing=True)
    keep = [0, 1, 2, 4, 5, 6, 7]
    logits = x @ router[keep].T
    p = np.exp(logits - logits.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    order = np.argsort(-logits, axis=1, kind="stable")[:, :2]
    np.testing.assert_array_equal(to_host(ids), np.array(keep)[order])
    assert (np.abs(_host(w) - np.take_along_axis(p, order, 1)) <= 2.0 ** -20).all()
    assert not torch.isnan(y).any()


def test_moe_ties_and_strides():
    """Equal router rows: the lower index.  Rows of x inside a wider buffer, odd offset."""
    q, torch = qz(), _t()
    case = (9, 64, 32, 12, 3, True, "bf16")
    x, xd, router, rd, st, dev = _moe_inputs(case)
    rd[5:9] = rd[4]
    rd[10] = rd[1]
    ids, p = mx4.route(x, rd.double().cpu().numpy(), 3, True)
    wide = torch.full((9, 80), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 7:71] = xd
    y, got, w = q.qz_mx4_moe(wide[:, 7:71], rd, *dev, 3, routing=True)
    np.testing.assert_array_equal(to_host(got), ids)
    assert torch.equal(y, q.qz_mx4_moe(xd, rd, *dev, 3))


def test_moe_nan_rows():
    """A token with a NaN (all its logits are NaN) takes the first experts and gives NaN; the
    others are as without it.  A NaN router row is chosen last."""
    q, torch = qz(), _t()
    case = (6, 64, 32, 8, 2, True, "bf16")
    x, xd, router, rd, st, dev = _moe_inputs(case)
    clean = q.qz_mx4_moe(xd, rd, *dev, 2)
    bad = xd.clone()
    bad[2, 5] = float("nan")
    y, ids, w = q.qz_mx4_moe(bad, rd, *dev, 2, routing=True)
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[2]).all() and list(to_host(ids)[2]) == [0, 1]
    r2 = rd.clone()
    r2[3] = float("nan")
    y, ids, w = q.qz_mx4_moe(xd, r2, *dev, 8, routing=True)
    assert (to_host(ids)[:, 7] == 3).all() and (to_host(w)[:, 7] == 0).all()
    assert not torch.isnan(y).any()


# --------------------------------------------------------------------- streams, graphs, a run
def test_streams_and_graph_replays():
    """The operators on a side stream and in a graph, replayed between eager work on new data."""
    q, torch = qz(), _t()
    case = (4, 200, 96, 8, 2, True, "bf16")     # rows that are copied to the workspace first
    x, xd, router, rd, st, dev = _moe_inputs(case)
    codes, scales = q.qz_mx4_quantize(torch.randn((300, 200), device="cuda"))

    def chain(inp):
        c, s = q.qz_mx4_quantize(inp)
        return (q.qz_mx4_linear(inp, codes, scales), q.qz_mx4_matmul(c, s, codes, scales, 200),
                q.qz_mx4_moe(inp, rd, *dev, 2))

    eager = chain(xd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = chain(xd)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    static = xd.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = chain(static)
    for seed in range(4):
        fresh = torch.randn((4, 200), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()
        static.copy_(fresh)
        g.replay()
        want = chain(fresh)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), seed


def test_two_streams_at_once():
    """The same operators on two streams at a time, each call with its own workspace."""
    q, torch = qz(), _t()
    x, xd, router, rd, st, dev = _moe_inputs((12, 512, 128, 16, 4, True, "bf16"))
    codes, scales = q.qz_mx4_quantize(torch.randn((2059, 3531), device="cuda"))
    big = torch.randn((1996, 3531), device="cuda").to(torch.bfloat16)     # split sums, padded rows

    def work():
        c, s = q.qz_mx4_quantize(big)
        return (q.qz_mx4_moe(xd, rd, *dev, 4), q.qz_mx4_linear(big, codes, scales),
                q.qz_mx4_matmul(c, s, codes, scales, 3531), q.qz_mx4_linear(big[:7], codes, scales))

    want = work()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(work())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))


def test_tensors_of_another_device_are_refused():
    q, torch = qz(), _t()
    x = torch.ones((2, 64), dtype=torch.bfloat16, device="cuda")
    c, s = q.qz_mx4_quantize(x)
    for bad in ((x, c.cpu(), s), (x, c, s.cpu()), (x.cpu(), c, s)):
        with pytest.raises(ValueError):
            q.qz_mx4_linear(*bad)
    with pytest.raises(ValueError):
        q.qz_mx4_linear(x, c, s, bias=torch.zeros(2))
    with pytest.raises(ValueError):
        q.qz_mx4_linear(x, c, s, out=torch.zeros((2, 2), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        q.qz_mx4_matmul(c, s.cpu(), c, s, 64)
    with pytest.raises(ValueError):
        q.qz_mx4_unpack(c, s.cpu(), 64)
    with pytest.raises(ValueError):
        q.qz_mx4_quantize(x, rule="least", colw=torch.ones(64))


def test_calibrate_quantise_and_use():
    """The operators as they are used together: Hessian, factors chosen under diag(H), the layer
    objective of the stored weights, and the layer run on its inputs."""
    q, torch = qz(), _t()
    rng = np.random.default_rng(3)
    x, xd = _bf16(rng.standard_t(4, (512, 256)) * np.where(rng.random(256) < 0.05, 20.0, 1.0))
    w = (rng.standard_normal((96, 256)) * 0.015).astype(np.float32)
    h = q.qz_build_hessian(xd, damp=0.01)
    f = {}
    for rule, colw in (("floor", None), ("least", h["diag"])):
        codes, scales, values = q.qz_mx4_quantize(to_dev(w), rule=rule, colw=colw, values=True)
        c, s, z = q.qz_mx4_unpack(codes, scales, 256)
        f[rule] = q.qz_objective(h["H"], to_dev(w), c, s, z, 32)
        want = objective.objective(_host(h["H"]), w, _host(values))
        assert abs(f[rule] - want) <= 1e-4 * want
        y = q.qz_mx4_linear(xd, codes, scales, out_dtype=torch.float32)
        v = _host(values)
        assert (np.abs(_host(y) - x @ v.T) <= _sum_bound(256, np.abs(x) @ np.abs(v).T, "f32", x @ v.T)).all()
    weighted = {r: (_host(h["diag"]) * (mx4.values(*mx4.quantize(w, r, c), 256) - w) ** 2).sum()
                for r, c in (("floor", None), ("least", to_host(h["diag"])))}
    assert weighted["least"] < weighted["floor"]


def test_timing_kinds_are_reported():
    q, torch = qz(), _t()
    q.qz_timing_read(reset=True)
    q.qz_timing_enable(True)
    c, s = q.qz_mx4_quantize(torch.randn((64, 64), device="cuda"))
    q.qz_mx4_matmul(c, s, c, s, 64)
    q.qz_timing_enable(False)
    t = q.qz_timing_read(reset=True)
    assert t["mx4_quantize"][0] == 1 and t["mx4_product"][0] == 1
