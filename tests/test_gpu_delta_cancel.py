"""The delta memory where a large old association is overwritten, in bf16 io:
y, dq and dk are then small differences of terms as large as the old memory.

Keys, queries and dy are unit vectors, alpha = 0 and theta = 1.  So a token
replaces one column of W (keys in the order of the columns), reads one that
was replaced before, and every product of a chunk picks single entries:
T = I, and what a result sums is W0's entry, the residual's (v less W0's
entry) and zeros.  Each of them is an fp32 value of size S = max |W0| after at
most one rounding, and a result adds at most six of them (a gradient meets two
memories, W and its adjoint), with the planes' dropped products below 2^-24 of
each: 16 u S covers that, beside half a step of bf16 of the result.  Factors
cut to 16 bits would be off by 2^-17 S on average, 8 times this bound.
"""
import numpy as np
import pytest

from delta_util import U16, U32
from oracle import delta_oracle as do

NAMES = ("k", "v", "q", "alpha", "theta", "W_in")
S = 2.0 ** 12


def problem(seed, H, N, d):
    rng = np.random.default_rng([seed, H, N, d])
    f32 = lambda x: x.astype(np.float32).astype(np.float64)
    unit = lambda at: np.eye(d)[at]
    f = {"k": unit(np.arange(N) % d)[None, None].repeat(H, 1),
         "q": unit(np.stack([[rng.integers(0, min(t, d - 1) + 1) for t in range(N)] for _ in range(H)]))[None],
         "v": rng.integers(-255, 256, (1, H, N, d)) / 128.0,       # bf16 values
         "alpha": np.zeros((1, H, N)), "theta": np.ones((1, H, N)),
         "W_in": f32(rng.uniform(-S, S, (1, H, d, d))),
         "dy": unit(rng.integers(0, d, (H, N)))[None]}
    return f


def tensors(f, device):
    import torch
    return {n: torch.from_numpy(x).to(torch.bfloat16 if n in ("k", "v", "q", "dy") else torch.float32).to(device)
            for n, x in f.items()}


def inside(name, got, want, half=U16):
    off = np.abs(got.double().cpu().numpy() - want)
    bound = half * np.abs(want) + 16 * U32 * S
    assert np.all(off <= bound), f"{name}: {np.max(off / bound):.2f} of the bound"


def test_the_problem_cancels():
    """On the CPU: y and most of dq are of v's size, and an fp32 recurrence stays within the bound."""
    import torch
    f = problem(1, 2, 64, 64)
    y, W = do.delta_forward(*(f[n] for n in NAMES))
    assert np.abs(y).max() <= 2.0 and np.abs(f["W_in"]).max() > 0.9 * S
    g = do.delta_backward(*(f[n] for n in NAMES), f["dy"])
    assert np.abs(g["q"]).max() > 1000 and np.median(np.abs(g["q"])) < 100   # overwritten columns beside old ones
    t = tensors(f, "cpu")
    w, ys = t["W_in"][0].clone(), []
    for i in range(64):
        k, v, q = (t[n][0, :, i].float() for n in ("k", "v", "q"))
        w = w + (v - (w * k[:, None]).sum(-1))[:, :, None] * k[:, None]
        ys.append((w * q[:, None]).sum(-1))
    inside("y", torch.stack(ys, 1)[None], y)


@pytest.mark.gpu
@pytest.mark.parametrize("recurrent", [False, True])
@pytest.mark.parametrize("H,N,d", [(2, 64, 64), (1, 32, 48), (2, 96, 96), (1, 128, 128), (2, 33, 33), (1, 100, 100)])
def test_y_of_an_overwritten_memory(H, N, d, recurrent):
    from test_learned_neural_amd import titans_mem as tmm
    f = problem(2, H, N, d)
    t = tensors(f, "cuda")
    y, W = tmm.delta_forward(*(t[n] for n in NAMES), force_recurrent=recurrent)
    yr, Wr = do.delta_forward(*(f[n] for n in NAMES))
    inside("y", y, yr)
    inside("W", W, Wr, U32)


@pytest.mark.gpu
@pytest.mark.parametrize("H,N,d", [(2, 64, 64), (1, 32, 48), (2, 96, 96), (1, 128, 128), (2, 33, 33), (1, 100, 100)])
def test_gradients_of_an_overwritten_memory(H, N, d):
    from test_learned_neural_amd import titans_mem as tmm
    f = problem(3, H, N, d)
    t = tensors(f, "cuda")
    got = tmm.delta_backward(*(t[n] for n in NAMES), dy=t["dy"])
    want = do.delta_backward(*(f[n] for n in NAMES), f["dy"])
    for name in ("q", "k"):
        inside(name, got[name], want[name])
