"""Host-only: the wrapper's four layouts of q, k and v."""
import pytest

from test_learned_neural_amd import titans_mem as tmm


def plan(q, k, sequences=None, last=None):
    import torch
    p = tmm._AttentionPlan(q, k, torch.float32, sequences, 0, 0, None, last)
    return (p.desc.B, p.desc.H, p.desc.Hk, p.desc.N, p.desc.d, p.desc.flags), p.keys, p.out, p.lse, p.back


def test_layouts():
    first, last = 0, tmm.FLAG_CHANNELS_LAST
    want = ((2, 5, 40), (2, 4, 5))
    a, b = plan((2, 4, 5, 10), (2, 2, 5, 10)), plan((2, 5, 4, 10), (2, 5, 2, 10), last=True)
    assert a[0] == (2, 4, 2, 5, 10, first) and b[0] == (2, 4, 2, 5, 10, last)
    assert a[1] == (2, 2, 5, 10) and b[1] == (2, 5, 2, 10) and a[2:4] == b[2:4] == want and a[4] == b[4] > 0
    want = ((7, 40), (4, 7))
    a, b = plan((7, 4, 10), (7, 2, 10), 3), plan((4, 7, 10), (2, 7, 10), 3, False)
    assert a[0] == (3, 4, 2, 7, 10, last) and b[0] == (3, 4, 2, 7, 10, first)
    assert a[1] == (7, 2, 10) and b[1] == (2, 7, 10) and a[2:4] == b[2:4] == want and a[4] == b[4] > 0
    assert plan((7, 4, 10), (7, 2, 10), 3, True) == a


def test_refusals():
    import torch
    z = torch.zeros
    with pytest.raises(ValueError, match="channels last"):
        tmm.attention(z(2, 5, 4), z(2, 5, 4), z(2, 5, 4), channels_last=True)
    with pytest.raises(ValueError):     # heads that do not share the tokens
        tmm.attention(z(2, 5, 4, 8), z(2, 6, 4, 8), z(2, 6, 4, 8), channels_last=True)
    with pytest.raises(ValueError):
        tmm.attention_backward(z(2, 5, 4, 8), z(2, 5, 2, 8), z(2, 5, 2, 8), z(2, 4, 32), z(2, 4, 5), z(2, 5, 32),
                               channels_last=True)
