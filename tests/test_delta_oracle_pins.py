"""The delta memory's oracle against things other than itself: finite
differences, torch's reverse mode, closed forms; and the chunk form that the
matrix-core kernels evaluate against the token recurrence."""
import numpy as np
import pytest

from delta_util import make
from oracle import delta_oracle as do


def test_full_step_stores_the_pair():
    # alpha = 0, theta = 1, |k| = 1: W_t k_t = v_t exactly, and directions orthogonal to k_t are untouched
    rng = np.random.default_rng(1)
    d = 12
    k = rng.standard_normal((1, 1, 1, d))
    k /= np.linalg.norm(k)
    v, W = rng.standard_normal((1, 1, 1, d)), rng.standard_normal((1, 1, d, d))
    z = np.zeros((1, 1, 1))
    y, W1 = do.delta_forward(k, v, k, z, z + 1, W)
    np.testing.assert_allclose(y, v, atol=1e-13)
    x = rng.standard_normal(d)
    x -= (x @ k[0, 0, 0]) * k[0, 0, 0]
    np.testing.assert_allclose(W1[0, 0] @ x, W[0, 0] @ x, atol=1e-12)


def test_forgetting_everything_leaves_the_last_pair():
    _, f = make(2, 2, 2, 1, 9, 8, "f32", edge="forget")
    _, W = do.delta_forward(f["k"], f["v"], f["q"], f["alpha"], f["theta"], f["W_in"])
    last = f["theta"][..., -1, None, None] * f["v"][:, :, -1, :, None] * f["k"][:, [0, 0], -1, None, :]
    np.testing.assert_allclose(W, last, atol=1e-14)


def test_matches_the_memory_rule_at_chunk_one_without_decay(oracle_mod):
    """alpha = 0: the residual is the undecayed one, so this is titans_mem_forward's linear memory at chunk 1, eta = 0."""
    _, f = make(3, 1, 3, 3, 40, 8, "f32", edge="keep")
    y, W = do.delta_forward(f["k"], f["v"], f["q"], f["alpha"], f["theta"], f["W_in"])
    r = lambda x: np.ascontiguousarray(x.reshape((3,) + x.shape[2:]))
    yr, Wr, _ = oracle_mod.forward(r(f["k"]), r(f["v"]), r(f["q"]), r(f["alpha"]), r(0 * f["alpha"]), r(f["theta"]),
                                   r(f["W_in"]).reshape(3, -1), np.zeros((3, 64)), d=8, hidden=0, n_layers=1, chunk=1)
    np.testing.assert_allclose(y.reshape(yr.shape), yr, rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(W.reshape(Wr.shape), Wr, rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("lengths", [None, [0, 5, 3]])
def test_gradient_matches_differences(lengths):
    B, H, Hk, N, d = 3, 2, 1, 5, 4
    _, f = make(4, B, H, Hk, N, d, "f32", lengths=lengths)
    f["alpha"][0, 0, 2] = 1.0
    names = ("k", "v", "q", "alpha", "theta", "W_in")
    g = do.delta_backward(*(f[n] for n in names), f["dy"], f["dW"], f["lengths"])

    def loss(x):
        y, W = do.delta_forward(*(x[n] for n in names), x["lengths"])
        live = np.ones((B, N)) if lengths is None else np.arange(N)[None] < f["lengths"][:, None]
        return np.sum(y * f["dy"] * live[:, None, :, None]) + np.sum(W * f["dW"])

    for name in names:
        it = np.random.default_rng(5).choice(f[name].size, min(12, f[name].size), replace=False)
        for i in it:
            e = 1e-5
            up, dn = ({**f, name: f[name].copy()} for _ in range(2))
            up[name].flat[i] += e
            dn[name].flat[i] -= e
            fd = (loss(up) - loss(dn)) / (2 * e)
            assert abs(fd - g[name].flat[i]) <= 1e-7 * max(1, abs(fd)), (name, i, fd, g[name].flat[i])


def test_chunk_form_equals_the_recurrence():
    """(I + B) F = V - diag(G) K W0^T, B[t,j] = D[t,j] (k_t.k_j) theta_j for j < t, and what follows from it."""
    N, d = 20, 6
    _, f = make(6, 1, 1, 1, N, d, "f32", resets=True)
    k, v, q, al, th, W0 = (f[n][0, 0] for n in ("k", "v", "q", "alpha", "theta", "W_in"))
    D = np.array([[np.prod(1 - al[j + 1:t + 1]) if j <= t else 0 for j in range(N)] for t in range(N)])
    G = np.cumprod(1 - al)
    F = np.linalg.solve(np.eye(N) + np.tril(D * (k @ k.T), -1) * th, v - G[:, None] * (k @ W0.T))
    U = th[:, None] * F
    y, W = do.delta_forward(*(f[n] for n in ("k", "v", "q", "alpha", "theta", "W_in")))
    np.testing.assert_allclose(G[:, None] * (q @ W0.T) + (D * (q @ k.T)) @ U, y[0, 0], atol=1e-12)
    np.testing.assert_allclose(G[-1] * W0 + (U * D[-1][:, None]).T @ k, W[0, 0], atol=1e-12)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("silu", [False, True])
def test_group_norm_against_torch(gated, silu):
    import torch
    rng = np.random.default_rng(7)
    x, w, b, z, do_ = (rng.standard_normal(s) for s in ((5, 3, 10), (3, 10), (3, 10), (5, 3, 10), (5, 3, 10)))
    t = [torch.from_numpy(a).requires_grad_() for a in (x, w, b, z)]
    n = torch.nn.functional.group_norm(t[0].reshape(5, 30), 3, t[1].reshape(-1), t[2].reshape(-1), 1e-3).reshape(5, 3, 10)
    act = torch.nn.functional.silu if silu else (lambda a: a)
    out = act(t[3]) * n if gated else act(n)
    np.testing.assert_allclose(do.group_norm(x, w, b, z if gated else None, silu, 1e-3), out.detach().numpy(), atol=1e-12)
    g = torch.autograd.grad(out, t if gated else t[:3], torch.from_numpy(do_))
    dx, dz, dw, db = do.group_norm(x, w, b, z if gated else None, silu, 1e-3, do_)
    for a, r in zip((dx, dw.sum(0), db.sum(0), dz), g):
        np.testing.assert_allclose(a, r.numpy(), atol=1e-11)
