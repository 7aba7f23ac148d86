"""Tensors that a delta memory or group norm call cannot do without are asked for by name (no GPU needed)."""
import pytest


def _delta():
    import torch
    B, H, Hk, N, d = 1, 2, 1, 3, 8
    return dict(k=torch.zeros(B, Hk, N, d), v=torch.zeros(B, H, N, d), q=torch.zeros(B, Hk, N, d),
                alpha=torch.zeros(B, H, N), theta=torch.zeros(B, H, N), W_in=torch.zeros(B, H, d, d))


@pytest.mark.parametrize("name", ["k", "v", "q", "alpha", "theta", "W_in"])
def test_delta_inputs(name):
    from test_learned_neural_amd import titans_mem as tmm
    a = {**_delta(), name: None}
    with pytest.raises(ValueError, match=f"^{name} "):
        tmm.delta_forward(*a.values())
    with pytest.raises(ValueError, match=f"^{name} "):
        tmm.delta_backward(*a.values(), dy=_delta()["v"])


def test_adjoints():
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    with pytest.raises(ValueError, match="^dy "):
        tmm.delta_backward(*_delta().values(), dy=None)
    x = torch.zeros(2, 3, 4, 8)
    with pytest.raises(ValueError, match="^dout "):
        tmm.group_norm_backward(x, None, None, None)
    for call in (lambda: tmm.group_norm(None), lambda: tmm.group_norm_backward(None, None, None, torch.zeros(2, 4, 24))):
        with pytest.raises(ValueError, match="^x "):
            call()
