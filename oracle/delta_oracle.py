"""Gated delta memory and group norm, fp64, from their definitions (numpy).

Token by token over [streams, ...] arrays; no code shared with the library.
Test, smoke and documentation use only.

    f_t = v_t - (1 - alpha_t) W_{t-1} k_t
    W_t = (1 - alpha_t) W_{t-1} + theta_t f_t k_t^T
    y_t = W_t q_t
"""
from __future__ import annotations

import numpy as np


def _per_head(x, H):
    return np.repeat(x, H // x.shape[1], axis=1) if x.shape[1] != H else x


def delta_forward(k, v, q, alpha, theta, W_in, lengths=None, states=False):
    """k, q [B,Hk,N,d], v [B,H,N,d], gates [B,H,N], W_in [B,H,d,d], all fp64.
    Returns (y, W), y zero past a length; with ``states`` also the list of
    the state before every token and after the last, and the residuals."""
    B, H, N, d = v.shape
    k, q = _per_head(k, H), _per_head(q, H)
    n = np.full(B, N) if lengths is None else np.clip(lengths, 0, N)
    W, y, f = W_in.copy(), np.zeros_like(v), np.zeros_like(v)
    kept = [W]
    for t in range(N):
        on = t < n
        if on.any():
            W = W.copy()
            Wd = (1 - alpha[on, :, t])[..., None, None] * W[on]
            f[on, :, t] = v[on, :, t] - np.einsum("bhij,bhj->bhi", Wd, k[on, :, t])
            W[on] = Wd + theta[on, :, t][..., None, None] * f[on, :, t][..., :, None] * k[on, :, t][..., None, :]
            y[on, :, t] = np.einsum("bhij,bhj->bhi", W[on], q[on, :, t])
        kept.append(W)
    return (y, W, kept, f) if states else (y, W)


def delta_backward(k, v, q, alpha, theta, W_in, dy, dW_out=None, lengths=None):
    """Adjoints of delta_forward's inputs for dy [B,H,N,d] and dW_out [B,H,d,d]
    (None = zero), by the reverse of the token recurrence."""
    B, H, N, d = v.shape
    Hk = k.shape[1]
    _, _, W, f = delta_forward(k, v, q, alpha, theta, W_in, lengths, states=True)
    k, q = _per_head(k, H), _per_head(q, H)
    n = np.full(B, N) if lengths is None else np.clip(lengths, 0, N)
    dW = np.zeros_like(W_in) if dW_out is None else dW_out.copy()
    g = {"k": np.zeros_like(v), "v": np.zeros_like(v), "q": np.zeros_like(v), "alpha": np.zeros_like(alpha),
         "theta": np.zeros_like(theta)}
    for t in reversed(range(N)):
        on = t < n
        if not on.any():
            continue
        kt, th, a, ft = k[on, :, t], theta[on, :, t], 1 - alpha[on, :, t], f[on, :, t]
        g["q"][on, :, t] = np.einsum("bhij,bhi->bhj", W[t + 1][on], dy[on, :, t])
        D = dW[on] + dy[on, :, t][..., :, None] * q[on, :, t][..., None, :]
        Dk = np.einsum("bhij,bhj->bhi", D, kt)
        df = th[..., None] * Dk
        g["theta"][on, :, t] = np.sum(ft * Dk, -1)
        g["v"][on, :, t] = df
        g["k"][on, :, t] = th[..., None] * np.einsum("bhij,bhi->bhj", D, ft) - \
            a[..., None] * np.einsum("bhij,bhi->bhj", W[t][on], df)
        dH = D - df[..., :, None] * kt[..., None, :]
        g["alpha"][on, :, t] = -np.sum(dH * W[t][on], (-1, -2))
        dW[on] = a[..., None, None] * dH
    for name in ("k", "q"):
        g[name] = g[name].reshape(B, Hk, H // Hk, N, d).sum(2)
    g["W_in"] = dW
    return g


def _sigmoid(z):
    return 1 / (1 + np.exp(-z))


def group_norm(x, weight=None, bias=None, gate=None, silu=True, eps=1e-5, dout=None):
    """x, gate, dout [..., d] with weight, bias broadcastable to x, fp64, a
    group along the last axis.  Returns out, or with dout the adjoints (x,
    gate or None, and weight's and bias's per element, for the caller to sum)."""
    w = np.ones(x.shape[-1]) if weight is None else weight
    b = np.zeros(x.shape[-1]) if bias is None else bias
    mean = x.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + eps)
    xh = (x - mean) * rstd
    n = xh * w + b
    z = n if gate is None else gate
    s = _sigmoid(z) if silu else np.ones_like(z)
    f = z * s
    if dout is None:
        return f if gate is None else f * n
    slope = s * (1 + z * (1 - s)) if silu else np.ones_like(z)
    dn = dout * (slope if gate is None else f)
    dxh = dn * w
    dx = rstd * (dxh - dxh.mean(-1, keepdims=True) - xh * (dxh * xh).mean(-1, keepdims=True))
    return dx, None if gate is None else dout * n * slope, dn * xh, dn
