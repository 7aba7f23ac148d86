"""The attention's gradient over tensors of more than 2^31 elements: the last tokens' is right.

Only the last tokens are not zero, and the window keeps the ones that are compared
among them (bounds in attention_util.py)."""
import pytest

from attention_util import backward_want, forward_want, make, near

pytestmark = pytest.mark.gpu

H, D, LIVE, SEEN, WINDOW = 16, 128, 260, 150, 64


def _check(part, out, lse, grad):
    """[H, LIVE, d] of each; the last SEEN tokens and all that they touch are among the live ones."""
    o, ob, l, lb = forward_want(part, "bf16", D ** -0.5, WINDOW)
    near("out", out[:, -SEEN:], o[:, -SEEN:], ob[:, -SEEN:])
    near("lse", lse[:, -SEEN:], l[:, -SEEN:], lb[:, -SEEN:])
    for name, t, (w, wb) in zip("qkv", grad, backward_want(part, "bf16", D ** -0.5, WINDOW)):
        near("d" + name, t[:, -SEEN:], w[:, -SEEN:], wb[:, -SEEN:])


def test_packed():
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    total = (1 << 20) + 77
    part = make(101, H, H, [LIVE], D, "bf16")[0]
    q, k, v, do = (torch.zeros(total, H, D, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    for t, x in zip((q, k, v, do), part):
        t[total - LIVE:] = torch.from_numpy(x).bfloat16().transpose(0, 1)
    off = torch.tensor([3, 40, total], dtype=torch.int32, device="cuda")
    out, lse = tmm.attention(q, k, v, offsets=off, window=WINDOW)
    g = tmm.attention_backward(q, k, v, out, lse, do.reshape(total, H * D), offsets=off, window=WINDOW)
    end = lambda t: t[total - LIVE:].reshape(LIVE, H, D).transpose(0, 1)  # noqa: E731
    _check(part, end(out), lse[:, total - LIVE:], [end(g[n]) for n in "qkv"])
    for n in "qkv":
        assert (g[n][:3] == 0).all()


def test_padded():
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    B, N = 3, 350001
    part = make(102, H, H, [LIVE], D, "bf16")[0]
    q, k, v = (torch.zeros(B, H, N, D, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    do = torch.zeros(B, N, H, D, device="cuda", dtype=torch.bfloat16)
    for t, x in zip((q, k, v, do.transpose(1, 2)), part):
        t[-1, :, N - LIVE:] = torch.from_numpy(x).bfloat16()
    n = torch.tensor([5, 0, N], dtype=torch.int32, device="cuda")
    do = do.reshape(B, N, H * D)
    out, lse = tmm.attention(q, k, v, lengths=n, window=WINDOW)
    g = tmm.attention_backward(q, k, v, out, lse, do, lengths=n, window=WINDOW)
    _check(part, out[-1, N - LIVE:].reshape(LIVE, H, D).transpose(0, 1), lse[-1, :, N - LIVE:],
           [g[x][-1, :, N - LIVE:] for x in "qkv"])
    for x in "qkv":
        assert (g[x][0, :, 5:] == 0).all() and (g[x][1] == 0).all()
