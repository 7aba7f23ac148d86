"""The attention beside the memory, and the projection behind both, as a block runs them.

input side -> delta memory and windowed attention -> group norm of the memory's
y, gated by the attention's out -> output projection and residual; its gradient
back through all of them; and packed prompts whose q, k and v a projection made.
Every stage's oracle starts from the values that the GPU stage before it left,
so a stage answers for its own error alone.
"""
import numpy as np
import pytest

from attention_util import H16, U, backward_want, forward_want, near
from oracle import attention_oracle as ao
from oracle import delta_oracle as do

pytestmark = pytest.mark.gpu


def _f64(*ts):
    return [t.double().cpu().numpy() for t in ts]


def test_block_forward_and_gradient():
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    B, N, D, H, d = 2, 150, 256, 4, 64
    g = torch.Generator(device="cuda").manual_seed(51)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = r(B, N, D).bfloat16()
    n = torch.tensor([150, 97], dtype=torch.int32, device="cuda")
    k, v, q, alpha, _, theta = tmm.input_side(x, (r(3, H * d, D) / 16).bfloat16(), r(3, H * d, 4) / 2,
                                              (r(3, H, D) / 16).bfloat16(), 0.5 * r(3, H), (0.1, 1.0, 1.0), H=H, d=d)
    W0, wo = r(B, H, d, d) / 8, (r(D, H * d) / 16).bfloat16()
    y, _ = tmm.delta_forward(k, v, q, alpha, theta, W0, lengths=n)
    kw = dict(lengths=n, window=40, prefix=4, scale=1.0)
    att, lse = tmm.attention(q, k, v, **kw)
    h = tmm.group_norm(y, gate=att, lengths=n)                 # channels last, as the attention's out is
    out = tmm.projection(h, wo, residual=x)
    # and back
    dout = r(B, N, D).bfloat16()
    dp = tmm.projection_backward(h, wo, dout)
    dn = tmm.group_norm_backward(y, None, None, dp["x"], gate=att, lengths=n)
    da = tmm.attention_backward(q, k, v, att, lse, dn["gate"], **kw)
    dm = tmm.delta_backward(k, v, q, alpha, theta, W0, dy=dn["x"], lengths=n)
    assert all(torch.isfinite(t).all() for t in (out, *da.values(), *dm.values(), *dp.values()))
    for b, m in enumerate(n.tolist()):
        part = tuple(t[b, :, :m].double().cpu().numpy() for t in (q, k, v)) + (
            dn["gate"][b, :m].reshape(m, H, d).transpose(0, 1).double().cpu().numpy(),)
        o, ob, l, lb = forward_want(part, "bf16", 1.0, 40, 4)
        near("att", att[b, :m].reshape(m, H, d).transpose(0, 1), o, ob)
        near("lse", lse[b, :, :m], l, lb)
        for name, (w, wb) in zip("qkv", backward_want(part, "bf16", 1.0, 40, 4)):
            near("d" + name, da[name][b, :, :m], w, wb)
        assert (att[b, m:] == 0).all() and (h[b, m:] == 0).all() and torch.equal(out[b, m:], x[b, m:])
    xs, ws, rs, dd = _f64(h.reshape(-1, H * d), wo, x.reshape(-1, D), dout.reshape(-1, D))
    want, z = ao.projection(xs, ws, None, rs)
    near("out", out.reshape(-1, D), want, 8 * U * 16 * (np.abs(xs) @ np.abs(ws).T) + (H16 + 4 * U) * np.abs(want) +
         4 * U * np.abs(rs))
    dx, dw, _ = ao.projection_backward(xs, ws, dd)
    near("dh", dp["x"].reshape(-1, H * d), dx, 8 * U * 16 * (np.abs(dd) @ np.abs(ws)) + (H16 + U) * np.abs(dx))
    near("dwo", dp["weight"], dw, 8 * U * 18 * (np.abs(dd).T @ np.abs(xs)))
    nr = do.group_norm(_f64(y.transpose(1, 2))[0], gate=_f64(att.reshape(B, N, H, d))[0])
    live = (np.arange(N)[None] < n.cpu().numpy()[:, None])[..., None, None]
    got = _f64(h.reshape(B, N, H, d))[0]
    assert np.all(np.abs(got - nr * live) <= H16 * np.abs(nr) + 64 * U * np.maximum(np.abs(nr), np.abs(_f64(
        att.reshape(B, N, H, d))[0])))


def test_packed_prompts_from_a_projection():
    """q, k and v as three projections leave them, tokens first, sequences one behind the other."""
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    D, H, Hk, d, sizes = 128, 6, 2, 32, [3, 0, 140, 1, 77]
    T = sum(sizes)
    g = torch.Generator(device="cuda").manual_seed(52)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x = r(T, D)
    q, k, v = (tmm.projection(x, (r(h * d, D) / 11)).reshape(T, h, d) for h in (H, Hk, Hk))
    at = np.concatenate([[0], np.cumsum(sizes)])
    off = torch.tensor(at, dtype=torch.int32, device="cuda")
    out, lse = tmm.attention(q, k, v, offsets=off)
    y = tmm.projection(out, (r(D, H * d) / 14), residual=x)
    assert y.shape == x.shape and torch.isfinite(y).all()
    for a, b in zip(at[:-1], at[1:]):
        if a < b:
            part = tuple(t[a:b].transpose(0, 1).double().cpu().numpy() for t in (q, k, v))
            o, ob, l, lb = forward_want(part, "bf16", d ** -0.5)
            near("out", out[a:b].reshape(b - a, H, d).transpose(0, 1), o, ob)
            near("lse", lse[:, a:b], l, lb)
