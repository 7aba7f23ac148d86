"""fp64 reference of the causal attention and of the projection (test oracle, numpy).

Token i of a sequence sees token j where j <= i and (window == 0 or
i - j < window or j < prefix).  Everything is formed in full, row by row of
what the definitions say; nothing is shared with the GPU path.
"""
import numpy as np


def seen(n, window=0, prefix=0, first=0):
    """[n - first, n] of bool: which tokens (columns) tokens first .. n - 1 see."""
    i, j = np.arange(first, n)[:, None], np.arange(n)[None]
    return (j <= i) & ((window == 0) | (i - j < window) | (j < prefix))


def weights(q, k, mask, scale):
    """(P, lse) of one head: q [m, d], k [n, d]; a row without keys has P = 0 and lse = -inf."""
    x = np.where(mask, (q @ k.T) * scale, -np.inf)
    top = x.max(1, initial=-np.inf, keepdims=True)
    e = np.where(mask, np.exp(x - np.where(np.isfinite(top), top, 0.0)), 0.0)
    total = e.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.log(total) + np.where(np.isfinite(top), top, 0.0)
    return e / np.where(total > 0, total, 1.0), lse[:, 0]


def attention(q, k, v, scale, window=0, prefix=0):
    """One sequence: q [H, n, d], k, v [Hk, n, d] -> out [H, n, d], lse [H, n]."""
    H, n, _ = q.shape
    mask = seen(n, window, prefix)
    out, lse = np.zeros(q.shape[:2] + v.shape[2:]), np.zeros((H, n))
    for h in range(H):
        kh = h // (H // k.shape[0])
        P, lse[h] = weights(q[h], k[kh], mask, scale)
        out[h] = P @ v[kh]
    return out, lse


def attention_backward(q, k, v, dout, scale, window=0, prefix=0):
    """One sequence's (dq, dk, dv)."""
    H, n, _ = q.shape
    mask = seen(n, window, prefix)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for h in range(H):
        kh = h // (H // k.shape[0])
        P, _ = weights(q[h], k[kh], mask, scale)
        dP = dout[h] @ v[kh].T
        dS = P * (dP - (P * dP).sum(1, keepdims=True))
        dq[h] = scale * dS @ k[kh]
        dk[kh] += scale * dS.T @ q[h]
        dv[kh] += P.T @ dout[h]
    return dq, dk, dv


def attention_step(q, k, v, scale, window=0, prefix=0):
    """The last m tokens of a sequence over all of it: q [H, m, d], k, v [Hk, n, d] -> out [H, m, d].

    New tokens before the first place (m > n) come out as zeros.
    """
    H, m, d = q.shape
    n = k.shape[1]
    out = np.zeros((H, m, v.shape[2]))
    live = min(m, n)
    if live:
        mask = seen(n, window, prefix, n - live)
        for h in range(H):
            kh = h // (H // k.shape[0])
            out[h, m - live:] = weights(q[h, m - live:], k[kh], mask, scale)[0] @ v[kh]
    return out


def silu(z):
    return z / (1 + np.exp(-z))


def silu_slope(z):
    s = 1 / (1 + np.exp(-z))
    return s * (1 + z * (1 - s))


def projection(x, weight, bias=None, residual=None, activation=False):
    """(out, z)."""
    z = x @ weight.T + (0.0 if bias is None else bias)
    out = silu(z) if activation else z
    return (out if residual is None else out + residual), z


def projection_backward(x, weight, dout, pre=None):
    """(dx, dweight, dbias); pre: what went into the activation, None without one."""
    dz = dout if pre is None else dout * silu_slope(pre)
    return dz @ weight, dz.T @ x, dz.sum(0)
