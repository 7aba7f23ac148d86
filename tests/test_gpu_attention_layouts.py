"""The layouts that the other tests do not run: padded rows channels last, packed ones heads first.

The same numbers in the other layout give the same bits, and one case of each is
held against the fp64 oracle (bounds in attention_util.py)."""
import numpy as np
import pytest

from attention_util import backward_want, forward_want, make, near, packed, padded

pytestmark = pytest.mark.gpu

#          H  Hk  sizes              d   io    window prefix
CASES = [(4, 2, [127, 129, 0, 1], 64, "bf16", 0, 0), (6, 2, [131, 70], 96, "f32", 50, 3), (3, 1, [200, 33], 33, "bf16", 0, 0),
         (2, 2, [300], 128, "f32", 0, 0), (8, 8, [400, 64], 64, "bf16", 100, 16), (5, 1, [90, 2], 7, "f32", 0, 0),
         (8, 4, [520], 128, "bf16", 0, 0)]


def _back(q, k, v, do, other, **kw):
    """(out, lse, gradients) of the usual layout, and of the other one with its gradients in the usual one."""
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    turn = lambda t: t.transpose(-2, -3).contiguous()  # noqa: E731
    got = []
    for x, last in (((q, k, v), None), (tuple(turn(t) for t in (q, k, v)), other)):
        out, lse = tmm.attention(*x, channels_last=last, **kw)
        g = tmm.attention_backward(*x, out, lse, do, channels_last=last, **kw)
        assert all(g[n].shape == t.shape for n, t in zip("qkv", x))
        got.append([out, lse] + [g[n] if last is None else turn(g[n]) for n in "qkv"])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    return got[1]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_padded_channels_last(case):
    import torch
    H, Hk, sizes, d, io, window, prefix = case
    N, nan = max(sizes) + 3, float("nan")
    parts = make(91, H, Hk, sizes, d, io)
    q, k, v, do = (padded(parts, i, N, io, nan) for i in range(4))
    do = do.transpose(1, 2).reshape(len(sizes), N, H * d).contiguous()
    n = torch.tensor(sizes, dtype=torch.int32, device="cuda")
    out, lse, *grad = _back(q, k, v, do, True, lengths=n, window=window, prefix=prefix)
    for b, p in enumerate(parts):
        m = sizes[b]
        assert all((t[b, :, m:] == 0).all() for t in grad) and (out[b, m:] == 0).all() and (lse[b, :, m:] == 0).all()
        if m:
            o, ob, l, lb = forward_want(p, io, d ** -0.5, window, prefix)
            near("out", out[b, :m].reshape(m, H, d).transpose(0, 1), o, ob)
            near("lse", lse[b, :, :m], l, lb)
            for name, t, (w, wb) in zip("qkv", grad, backward_want(p, io, d ** -0.5, window, prefix)):
                near("d" + name, t[b, :, :m], w, wb)
    full = [t[:1, :, :max(m, 1)].contiguous() for t, m in ((q, sizes[0]), (k, sizes[0]), (v, sizes[0]))]
    _back(*full, do[:1, :max(sizes[0], 1)].contiguous(), True, window=window, prefix=prefix)       # no lengths


@pytest.mark.parametrize("case", CASES, ids=str)
def test_packed_heads_first(case):
    import torch
    H, Hk, sizes, d, io, window, prefix = case
    first, total, nan = 5, 5 + sum(sizes) + 4, float("nan")
    parts = make(92, H, Hk, sizes, d, io)
    q, k, v, do = (packed(parts, i, total, first, io, nan) for i in range(4))
    at = np.concatenate([[first], first + np.cumsum(sizes)])
    off = torch.tensor(at, dtype=torch.int32, device="cuda")
    out, lse, *grad = _back(q, k, v, do.reshape(total, H * d), False, offsets=off, window=window, prefix=prefix)
    outside = torch.ones(total, dtype=torch.bool, device="cuda")
    outside[first:at[-1]] = False
    assert all((t[outside] == 0).all() for t in grad) and (out[outside] == 0).all()
    for s, p in enumerate(parts):
        a, b = int(at[s]), int(at[s + 1])
        if a < b:
            o, ob, l, lb = forward_want(p, io, d ** -0.5, window, prefix)
            near("out", out[a:b].reshape(b - a, H, d).transpose(0, 1), o, ob)
            near("lse", lse[:, a:b], l, lb)
            for name, t, (w, wb) in zip("qkv", grad, backward_want(p, io, d ** -0.5, window, prefix)):
                near("d" + name, t[a:b].transpose(0, 1), w, wb)
