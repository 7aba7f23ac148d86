"""One row and a weight of 2^29 numbers: the forward call and the gradient against torch, where single products are exact."""
import pytest

from attention_util import H16, U

pytestmark = pytest.mark.gpu


def test_one_row_of_many_channels():
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    K, O = 8192, 65536
    g = torch.Generator(device="cuda").manual_seed(61)
    x = torch.randn(1, K, generator=g, device="cuda").bfloat16()
    w = torch.randn(O, K, generator=g, device="cuda").bfloat16()
    dout = torch.randn(1, O, generator=g, device="cuda").bfloat16()
    out = tmm.projection(x, w).double()[0]
    got = tmm.projection_backward(x, w, dout)
    for a in range(0, O, 4096):      # 8 u sqrt(n) of the terms for a sum of n, half a step of bf16 for out
        part = w[a:a + 4096].double()
        want, size = (part @ x[0].double()), part.abs() @ x[0].double().abs()
        assert ((out[a:a + 4096] - want).abs() <= 8 * U * K ** 0.5 * size + (H16 + U) * want.abs()).all()
        assert torch.equal(got["weight"][a:a + 4096], dout[0, a:a + 4096, None].float() * x.float())
    dx = torch.zeros(K, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(dx)
    for a in range(0, O, 4096):
        part, d = w[a:a + 4096].double(), dout[0, a:a + 4096].double()
        dx += d @ part
        size += d.abs() @ part.abs()
    assert ((got["x"][0].double() - dx).abs() <= 8 * U * O ** 0.5 * size + (H16 + U) * dx.abs()).all()
    assert torch.equal(got["bias"], dout[0].float())
