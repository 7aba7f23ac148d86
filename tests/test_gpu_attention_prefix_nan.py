"""A NaN or an infinity behind the persistent tokens, within what a tile of the prefix holds, stays near its token.

A workgroup has 128 queries and reads whole tiles of 64 keys where its first query's window begins, so a token can
reach queries that it is out of the window of by up to 127 + 63 tokens; tiles before that are read for the
persistent tokens alone."""
import pytest

from attention_util import dtype

pytestmark = pytest.mark.gpu

NEAR = 127 + 63


def _inputs(io, N=900, H=4, Hk=2, d=64):
    import torch
    g = torch.Generator(device="cuda").manual_seed(121)
    return [torch.randn(s, generator=g, device="cuda").to(dtype(io))
            for s in ((1, H, N, d), (1, Hk, N, d), (1, Hk, N, d), (1, N, H * d))]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("window,prefix,at", [(100, 5, 10), (100, 5, 5), (1, 1, 31), (200, 63, 63), (64, 70, 100), (37, 33, 60)])
def test_prompt_and_gradient(window, prefix, at, io, bad):
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    q, k, v, do = _inputs(io)
    kw = dict(window=window, prefix=prefix)
    out, lse = tmm.attention(q, k, v, **kw)
    grad = tmm.attention_backward(q, k, v, out, lse, do, **kw)
    w = v.clone()
    w[0, 1, at, 3] = bad
    got, stat = tmm.attention(q, k, w, **kw)
    far = at + window + NEAR
    assert torch.equal(stat, lse) and torch.equal(got[0, far:], out[0, far:]) and torch.equal(got[0, :, :128], out[0, :, :128])
    assert not torch.isfinite(got[0, at:at + window, 128 + 3]).any()
    # the gradient at what the forward call left: far queries' is what it was, whichever of k and v is bad
    assert torch.equal(tmm.attention_backward(q, k, w, out, lse, do, **kw)["q"][0, :, far:], grad["q"][0, :, far:])
    w = k.clone()
    w[0, 1, at, 3] = bad
    assert torch.equal(tmm.attention_backward(q, w, v, out, lse, do, **kw)["q"][0, :, far:], grad["q"][0, :, far:])


@pytest.mark.parametrize("which", ["q", "dout"])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_gradient_of_keys(io, which):
    """A far query's NaN: the persistent tokens see it, and the 31 behind them at most share their operands."""
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    q, k, v, do = _inputs(io)
    at, window, prefix = 700, 100, 5
    kw = dict(window=window, prefix=prefix)
    out, lse = tmm.attention(q, k, v, **kw)
    want = tmm.attention_backward(q, k, v, out, lse, do, **kw)
    bad, other = q.clone(), do.clone()
    if which == "q":
        bad[0, 0, at, 3] = float("nan")
    else:
        other[0, at, 3] = float("nan")
    got = tmm.attention_backward(bad, k, v, out, lse, other, **kw)
    for name in "kv":
        a, b = got[name][0], want[name][0]
        assert torch.equal(a[1], b[1])                                             # the other key head
        assert torch.equal(a[0, prefix + 31:at - window - 255], b[0, prefix + 31:at - window - 255])
        assert torch.equal(a[0, at + 256:], b[0, at + 256:])
        assert torch.isnan(a[0, :prefix]).any(-1).all() and torch.isnan(a[0, at - window + 1:at + 1]).any(-1).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,window,prefix,at", [(1, 100, 5, 10), (3, 64, 1, 31), (2, 200, 40, 50)])
def test_step(n, window, prefix, at, io):
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    q, k, v, _ = _inputs(io)
    q, ln = q[:, :, -n:].contiguous(), torch.tensor([900], dtype=torch.int32, device="cuda")
    want = tmm.attention_step(q, k, v, ln, window=window, prefix=prefix)
    v[0, 1, at, 3] = float("nan")
    assert torch.equal(tmm.attention_step(q, k, v, ln, window=window, prefix=prefix), want)
