"""The gradient where scores are hundreds apart: weights are formed from lse, and come out 0, 1 and between.

Bounds in attention_util.py: the weights' error has the scores' (8 u sqrt(d) + 8 u of the largest) and lse's (4 u of it).
Weights below 2^-126 have no fp32 numbers: up to 300 of them, at |dP - D| < 2^8, scale |q| or scale |k| < 2^5 and
|dout| < 2^3 an element, put a gradient off by less than 2^-100."""
import numpy as np
import pytest

from attention_util import backward_want, dtype, forward_want, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("window,prefix", [(0, 0), (90, 7)])
def test_gradient(io, window, prefix):
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    rng = np.random.default_rng(131)
    q, k, v, do = (torch.from_numpy(rng.standard_normal((1, 2, 300, 64)) * s).to(dtype(io)).cuda() for s in (40, 1, 1, 1))
    k[:, :, 100:200] *= 40
    part = tuple(t[0].double().cpu().numpy() for t in (q, k, v, do))
    kw = dict(window=window, prefix=prefix)
    out, lse = tmm.attention(q, k, v, **kw)
    o, ob, l, lb = forward_want(part, io, 0.125, window, prefix)
    near("out", out[0].reshape(300, 2, 64).transpose(0, 1), o, ob)
    near("lse", lse[0], l, lb)
    grad = tmm.attention_backward(q, k, v, out, lse, do.transpose(1, 2).reshape(1, 300, 128).contiguous(), **kw)
    for name, (w, wb) in zip("qkv", backward_want(part, io, 0.125, window, prefix)):
        near("d" + name, grad[name][0], w, wb + 2.0 ** -100)
