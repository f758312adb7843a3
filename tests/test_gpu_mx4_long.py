"""GPU: products with MX4 weights whose rows need several fetches of factors (a tile kernel holds 64
blocks of a row at a time), exact in every output.  The factors differ from one run of 64 blocks to
the next, so that a sum over the factors of another run is another sum."""
import pytest

from gpu_util import qz

pytestmark = pytest.mark.gpu

# n, d_i, d_o; d_i a multiple of 128, so that factors are copied by words.  tests/test_mx4_plan.py
# holds which kernel each one reaches, and that a split has 70 stages or more.
LONG_LINEAR = [
    (2054, 4480, 4296), (1158, 8832, 4354), (1284, 4480, 3687), (514, 13184, 3600), (2439, 4480, 3079),
    (1284, 13184, 1802), (1025, 4480, 3600), (262, 13184, 3687), (388, 5248, 4383), (129, 13440, 4122)]
STEPS = [0, 4, 1, 5, 2]   # exponents of the runs


def _stored(rows, cols, gen):
    """(codes, scales, values in 64 bits) of a random matrix: multiples of 1/4."""
    import torch
    codes = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, device="cuda", generator=gen)
    scales = torch.randint(126, 129, (rows, cols // 32), dtype=torch.uint8, device="cuda", generator=gen)
    run = torch.arange(cols // 32, device="cuda") // 64 % len(STEPS)
    scales += torch.tensor(STEPS, dtype=torch.uint8, device="cuda")[run]
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    table = torch.cat([table, -table])
    v = table[torch.stack([codes & 15, codes >> 4], -1).flatten(1).int()]
    return codes, scales, v * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)


@pytest.mark.parametrize("n,d_i,d_o", LONG_LINEAR)
def test_factors_of_many_runs(n, d_i, d_o):
    """x in -3 .. 3 (exact in E2M1 too): sums of multiples of 1/4 below 2^22, exact in fp32."""
    import torch
    q = qz()
    gen = torch.Generator("cuda").manual_seed(n)
    codes, scales, w = _stored(d_o, d_i, gen)
    x = torch.randint(-3, 4, (n, d_i), device="cuda", generator=gen).double()
    assert float((x.abs() @ w.abs().T).max()) < 2.0 ** 22
    want = x @ w.T
    xd = x.to(torch.bfloat16)
    for _ in range(3):
        got = q.qz_mx4_linear(xd, codes, scales, out_dtype=torch.float32)
        assert torch.equal(got.double(), want)
    xc, xs = q.qz_mx4_quantize(xd)
    got = q.qz_mx4_matmul(xc, xs, codes, scales, d_i, out_dtype=torch.float32)
    assert torch.equal(got.double(), want)


@pytest.mark.parametrize("n,d_i,d_o", [(262, 13184, 3687), (388, 5248, 4383)])
def test_long_products_in_a_graph(n, d_i, d_o):
    """Split sums and a single launch, replayed between eager calls on other data."""
    import torch
    q = qz()
    gen = torch.Generator("cuda").manual_seed(d_i)
    codes, scales, _ = _stored(d_o, d_i, gen)
    static = torch.zeros((n, d_i), dtype=torch.bfloat16, device="cuda")

    def chain(x):
        xc, xs = q.qz_mx4_quantize(x)
        return q.qz_mx4_linear(x, codes, scales), q.qz_mx4_matmul(xc, xs, codes, scales, d_i)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = chain(static)
    for _ in range(4):
        x = torch.randn((n, d_i), device="cuda", generator=gen).to(torch.bfloat16)
        want = chain(x)
        static.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
