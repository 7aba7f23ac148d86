"""A bf16 gradient that is infinite, or becomes so as it is rounded: the weight's gradient is infinite, and no NaN, where
every term has one sign; other rows of it are what they were."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), 3.3895313892515355e38])
@pytest.mark.parametrize("M,K,O", [(5, 16, 24), (300, 33, 40), (5000, 64, 520)])
def test_weight_gradient(M, K, O, bad):
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    g = torch.Generator(device="cuda").manual_seed(141)
    x = torch.rand(M, K, generator=g, device="cuda").add(0.5).bfloat16()
    w = torch.randn(O, K, generator=g, device="cuda").bfloat16()
    do, pre = (torch.randn(M, O, generator=g, device="cuda").bfloat16() for _ in range(2))
    pre[M // 2, 7] = 1.5               # SiLU's slope is 1.04: the largest number becomes infinite
    want = tmm.projection_backward(x, w, do, pre=pre, activation=tmm.ACT_SILU)
    do[M // 2, 7] = bad
    got = tmm.projection_backward(x, w, do, pre=pre, activation=tmm.ACT_SILU)
    sign = 1 if bad > 0 else -1
    assert torch.equal(got["weight"][7], torch.full((K,), sign * float("inf"), device="cuda"))
    rest = torch.arange(O, device="cuda") != 7
    assert torch.equal(got["weight"][rest], want["weight"][rest]) and torch.equal(got["bias"][rest], want["bias"][rest])
