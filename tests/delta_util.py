"""Inputs, oracle runs and comparisons shared by the delta memory's tests.

Tolerances.  u = 2^-24 is half a step of fp32, 2^-8 half a step of bf16
relative to the value.  One token's update of a state element is a dot product
over d (at most d roundings of terms whose sum's norm is that of the row) and a
handful more; a rounding's effect decays or stays over the later tokens.  The
roundings' signs are taken as independent, so after N tokens a norm is off by
a small multiple of u sqrt(d N) relative to the norm of what was summed:
16 u sqrt(d N) is asked, with N at least 16.  A chunked kernel sums over the
chunk's tokens in another order, with the same count.  The gradient runs the
recurrence forward and back and multiplies the two, so it gets four times
that.  A stored io value adds its own half step of bf16.
"""
import math

import numpy as np

U32, U16 = 2.0 ** -24, 2.0 ** -8


def tol32(N, d):
    return 16 * U32 * math.sqrt(d * max(N, 16))


def rounded(x, io):
    """fp64 values as the io type holds them."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16 if io == "bf16" else torch.float32)
    return t, t.double().numpy()


def make(seed, B, H, Hk, N, d, io, ragged=False, resets=False, edge=None, lengths=None):
    """(device-typed CPU tensors, fp64 arrays) of one problem."""
    import torch
    rng = np.random.default_rng([seed, B, H, Hk, N, d])
    t, f = {}, {}
    for name in ("k", "q"):
        x = rng.standard_normal((B, Hk, N, d))
        x = x / (1 + np.exp(-x))
        x /= np.maximum(np.sqrt((x * x).sum(-1, keepdims=True)), 1e-6)
        t[name], f[name] = rounded(x, io)
    t["v"], f["v"] = rounded(rng.standard_normal((B, H, N, d)), io)
    t["dy"], f["dy"] = rounded(rng.standard_normal((B, H, N, d)), io)
    alpha = 0.1 / (1 + np.exp(-rng.standard_normal((B, H, N))))
    theta = 1 / (1 + np.exp(-rng.standard_normal((B, H, N))))
    if resets:
        alpha[rng.random((B, H, N)) < 0.03] = 1.0
    if edge == "keep":
        alpha[:] = 0.0
    elif edge == "forget":
        alpha[:] = 1.0
    elif edge == "still":
        theta[:] = 0.0
    elif edge == "full":
        alpha[:], theta[:] = 0.0, 1.0
    elif edge == "strong":      # decays far below fp32 within a few tokens
        alpha = 1 - 10.0 ** rng.uniform(-30, -1, (B, H, N))
    for name, x in (("alpha", alpha), ("theta", theta), ("W_in", rng.standard_normal((B, H, d, d)) / math.sqrt(d)),
                    ("dW", rng.standard_normal((B, H, d, d)))):
        t[name], f[name] = rounded(x, "f32")
    n = None
    if lengths is not None:
        n = np.asarray(lengths, np.int32)
    elif ragged:
        n = rng.permutation(np.round(np.linspace(0, N, B)).astype(np.int32)) if B > 1 else np.array([N // 2], np.int32)
    t["lengths"] = None if n is None else torch.from_numpy(n)
    f["lengths"] = n
    return t, f


def cuda(t):
    return {k: None if x is None else x.cuda() for k, x in t.items()}


def check(name, got, want, io, tol, rows=True):
    """got (tensor) against want (fp64): per leading stream norm-wise, and per row of the last axis relative to the
    larger of the row's own norm and the stream's mean row."""
    import torch
    g = got.double().cpu().numpy()
    assert g.shape == want.shape, (name, g.shape, want.shape)
    if not g.size:
        return 0.0
    assert np.isfinite(g).all(), name
    half = U16 if got.dtype == torch.bfloat16 else 0.0
    bound = tol + half
    S = g.shape[0] * g.shape[1]
    d = (g - want).reshape(S, -1)
    w = want.reshape(S, -1)
    norm = np.maximum(np.sqrt((w * w).sum(1)), 1e-30)
    e = np.sqrt((d * d).sum(1)) / norm
    assert e.max() <= bound, f"{name}: stream error {e.max():.3e} over {bound:.3e}"
    if rows and g.ndim >= 4:
        dr, wr = (np.sqrt((x.reshape(S, -1, g.shape[-1]) ** 2).sum(-1)) for x in (d, w))
        floor = np.maximum(np.sqrt((wr * wr).mean(1, keepdims=True)), 1e-30)
        er = dr / np.maximum(wr, floor)
        assert er.max() <= 4 * bound, f"{name}: row error {er.max():.3e} over {4 * bound:.3e}"
    return float(e.max())
