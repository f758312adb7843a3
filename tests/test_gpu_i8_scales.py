"""GPU: the scales of qz_i8_quantize beside those that torch's own operations give."""
import pytest

from gpu_util import qz

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales_as_torch_divides(dtype):
    """max |x| / 127 in torch on this GPU is a product with 1 / 127 rounded to 32 bits: the same scales, and so the
    same codes for whoever quantizes there with them."""
    import torch
    q = qz()
    x = torch.randn((4000, 321), device="cuda").mul_(torch.rand((4000, 1), device="cuda") * 9)
    x = x.to({"bf16": torch.bfloat16, "f32": torch.float32}[dtype])
    c, s = q.qz_i8_quantize(x)
    want = x.float().abs().amax(1) / 127.0
    assert torch.equal(s, want)
    code = (x.double() / want.double()[:, None]).round().clamp(-127, 127).to(torch.int8)
    assert torch.equal(c[:, :321], code)
