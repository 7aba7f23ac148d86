"""Gradients through the gated delta memory against the fp64 oracle (itself
pinned to differences), and against differences of the GPU's own forward."""
import numpy as np
import pytest

from delta_util import check, cuda, make, tol32
from oracle import delta_oracle as do

pytestmark = pytest.mark.gpu

NAMES = ("k", "v", "q", "alpha", "theta", "W_in")

#         B  H  Hk N    d    io      ragged resets edge   carry
SHAPES = [(1, 1, 1, 1, 64, "bf16", False, False, None, False),
          (2, 2, 1, 2, 1, "f32", False, False, None, True),
          (1, 3, 3, 7, 16, "bf16", False, False, None, True),
          (3, 2, 2, 31, 33, "f32", True, True, None, False),
          (2, 2, 2, 32, 64, "bf16", False, False, None, False),
          (2, 4, 2, 33, 64, "f32", False, False, None, True),
          (2, 4, 1, 64, 128, "bf16", False, False, None, True),
          (3, 6, 2, 65, 100, "f32", True, True, None, True),
          (3, 6, 2, 65, 100, "bf16", True, True, None, True),
          (2, 3, 3, 129, 63, "bf16", True, False, None, False),
          (2, 2, 1, 100, 128, "f32", True, True, None, True),
          (2, 3, 1, 100, 80, "bf16", False, True, None, True),
          (5, 2, 2, 200, 64, "bf16", True, True, None, True),
          (1, 2, 2, 300, 48, "f32", False, False, None, False),
          (1, 2, 2, 70, 64, "bf16", False, False, "keep", True),
          (1, 2, 2, 70, 64, "f32", False, False, "forget", True),
          (1, 2, 2, 70, 64, "f32", False, False, "still", True),
          (1, 2, 2, 70, 80, "f32", False, False, "full", True),
          (2, 2, 2, 70, 64, "f32", False, False, "strong", True)]


def _run(t, carry=True, **kw):
    from test_learned_neural_amd import titans_mem as tmm
    return tmm.delta_backward(*(t[n] for n in NAMES), dy=t["dy"], dW_out=t["dW"] if carry else None,
                              lengths=t["lengths"], **kw)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients(shape):
    B, H, Hk, N, d, io, ragged, resets, edge, carry = shape
    t, f = make(31, B, H, Hk, N, d, io, ragged, resets, edge)
    got = _run(cuda(t), carry)
    want = do.delta_backward(*(f[n] for n in NAMES), f["dy"], f["dW"] if carry else None, f["lengths"])
    tol = 4 * tol32(N, d)
    for name in NAMES:
        x = got[name]
        if f["lengths"] is not None and name not in ("W_in",):
            for b, n in enumerate(f["lengths"]):
                assert (x[b, :, max(0, n):] == 0).all(), name
        print(shape, name, check(name, x, want[name], io, tol), flush=True)


def test_what_lies_past_a_length_is_not_read():
    import torch
    t, f = make(32, 4, 4, 2, 70, 64, "bf16", lengths=[0, 70, 1, 33])
    g = cuda(t)
    want = _run(g)
    for name in ("k", "v", "q", "alpha", "theta", "dy"):
        for b, n in enumerate(f["lengths"]):
            g[name][b, :, n:] = float("nan")
    got = _run(g)
    for name in NAMES:
        assert torch.equal(got[name], want[name]), name
    assert torch.equal(got["W_in"][0], g["dW"][0])


def test_no_tokens():
    import torch
    t, _ = make(33, 2, 2, 1, 0, 64, "f32")
    g = cuda(t)
    got = _run(g)
    assert torch.equal(got["W_in"], g["dW"]) and got["k"].shape == (2, 1, 0, 64)
    assert (_run(g, carry=False)["W_in"] == 0).all()


def test_against_differences_of_the_forward():
    """Directional differences of the fp32 forward, in both directions of a random line."""
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    B, H, Hk, N, d = 1, 2, 1, 48, 32
    t, f = make(34, B, H, Hk, N, d, "f32")
    g = cuda(t)
    grad = _run(g)
    gen = torch.Generator(device="cuda").manual_seed(1)

    def loss(x):
        y, W = tmm.delta_forward(*(x[n] for n in NAMES))
        return float((y.double() * g["dy"].double()).sum() + (W.double() * g["dW"].double()).sum())

    for name in NAMES:
        u = torch.randn(g[name].shape, generator=gen, device="cuda")
        h = 2.0 ** -7 * float(g[name].norm() / u.norm())
        fd = (loss({**g, name: g[name] + h * u}) - loss({**g, name: g[name] - h * u})) / (2 * h)
        an = float((grad[name].double() * u.double()).sum())
        # the third derivative's term h^2 and the forward's rounding over h, both relative to |grad| |u|
        scale = float(grad[name].double().norm() * u.double().norm())
        assert abs(fd - an) <= 1e-2 * scale, (name, fd, an, scale)


def test_same_bits_streams_and_replayed_graphs():
    import torch
    t, _ = make(35, 2, 4, 2, 150, 64, "bf16", ragged=True)
    g = cuda(t)
    want = _run(g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = _run(g)
    s.synchronize()
    assert all(torch.equal(want[n], got[n]) for n in NAMES)
    x = {n: None if v is None else v.clone() for n, v in g.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _run(x)
    for rep in range(4):
        x["dy"].copy_(g["dy"] * (rep + 1))
        want = _run({**g, "dy": g["dy"] * (rep + 1)})
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(want[n], out[n]) for n in NAMES)


@pytest.mark.parametrize("B,H,Hk,N,d,io,lengths", [
    (2, 2, 1, 70, 65, "f32", None), (2, 2, 1, 70, 67, "bf16", [70, 33]), (2, 4, 2, 99, 96, "f32", [99, 64]),
    (2, 4, 2, 99, 96, "bf16", None), (1, 2, 2, 65, 92, "bf16", None), (1, 2, 1, 65, 88, "bf16", [64]),
    (2, 2, 2, 40, 97, "f32", None), (40, 4, 2, 40, 84, "f32", None), (40, 4, 2, 40, 96, "bf16", None)])
def test_widths_between_64_and_128(B, H, Hk, N, d, io, lengths):
    t, f = make(61, B, H, Hk, N, d, io, resets=True, lengths=lengths)
    got = _run(cuda(t))
    want = do.delta_backward(*(f[n] for n in NAMES), f["dy"], f["dW"], f["lengths"])
    for name in NAMES:
        check(name, got[name], want[name], io, 4 * tol32(N, d))
