"""Inputs, oracle runs and bounds shared by the attention's tests.

Bounds, element by element, with u = 2^-24 (half a step of fp32) and h = 2^-8
(of bf16; 0 for fp32 tensors):

- A score is a sum of d products.  bf16 products are exact; of an fp32 one, the
  three bf16 planes leave out less than 4 u.  The sum's roundings are taken as
  independent: x is off by at most e_x = 8 u sqrt(d) times scale |q| |k|, where
  the largest of the sequence is taken, and the exponent's own rounding adds
  4 u times the span of the scores.  A weight is off by that relative to itself,
  the sum of n of them by sqrt(n) u more: e = e_x + 4 u span + 4 u sqrt(n) + 16 u.
- out = sum of P v: e + h (the weights that meet v) times sum P |v|, and h |out|
  for the result.  lse is off by e and 4 u |lse|.
- dS = P (dP - D): dP is off by 8 u sqrt(d) |dout| |v|, D by as much and by what
  the stored out is off by, |dout| . (h sum P |v| + h |out| + e sum P |v|); P by
  e relative to itself, and dS is rounded to h of itself before the products.
  dq, dk and dv sum those over rows or columns, with sqrt(n) u of the sum's
  terms for their own roundings, and end in h of themselves.
"""
import numpy as np

from oracle import attention_oracle as ao

U, H16 = 2.0 ** -24, 2.0 ** -8


def rounded(x, io):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16 if io == "bf16" else torch.float32)
    return t, t.double().numpy()


def make(seed, H, Hk, sizes, d, io, spread=1.0):
    """Per sequence fp64 (q [H, n, d], k, v [Hk, n, d], dout [H, n, d]), already rounded to the io type."""
    rng = np.random.default_rng([seed, H, Hk, d, *sizes])
    draw = lambda *s: rounded(spread * rng.standard_normal(s), io)[1]  # noqa: E731
    return [(draw(H, n, d), draw(Hk, n, d), draw(Hk, n, d), draw(H, n, d)) for n in sizes]


def dtype(io):
    import torch
    return torch.bfloat16 if io == "bf16" else torch.float32


def padded(parts, which, N, io, fill=0.0, device="cuda"):
    """[B, heads, N, d] of one tensor of make()'s sequences, `fill` past their lengths."""
    import torch
    heads, _, d = parts[0][which].shape
    t = torch.full((len(parts), heads, N, d), fill, dtype=torch.float64)
    for b, p in enumerate(parts):
        t[b, :, :p[which].shape[1]] = torch.from_numpy(p[which])
    return t.to(dtype(io)).to(device)


def packed(parts, which, total, first, io, fill=0.0, device="cuda"):
    """[total, heads, d]: the sequences one behind the other from row `first` on."""
    import torch
    heads, _, d = parts[0][which].shape
    t = torch.full((total, heads, d), fill, dtype=torch.float64)
    at = first
    for p in parts:
        n = p[which].shape[1]
        t[at:at + n] = torch.from_numpy(p[which]).transpose(0, 1)
        at += n
    return t.to(dtype(io)).to(device)


def _norms(q, k, v, do=None):
    f = lambda t: np.sqrt((t * t).sum(-1)).max() if t.size else 0.0  # noqa: E731
    return f(q), f(k), f(v), 0.0 if do is None else f(do)


def _weight_error(q, k, n, scale):
    d = q.shape[-1]
    nq, nk, _, _ = _norms(q, k, k)
    span = scale * nq * nk
    return (8 * U * np.sqrt(d) + 8 * U) * span + 4 * U * np.sqrt(max(n, 1)) + 16 * U


def forward_want(part, io, scale, window=0, prefix=0):
    """(out, its bound, lse, its bound) of one sequence, heads first."""
    q, k, v = part[:3]
    Hh, n, _ = q.shape
    h = H16 if io == "bf16" else 0.0
    out, lse = ao.attention(q, k, v, scale, window, prefix)
    e = _weight_error(q, k, n, scale)
    bound = np.zeros_like(out)
    mask = ao.seen(n, window, prefix)
    for i in range(Hh):
        kh = i // (Hh // k.shape[0])
        P, _ = ao.weights(q[i], k[kh], mask, scale)
        bound[i] = (2 * e + h) * (P @ np.abs(v[kh])) + (h + U) * np.abs(out[i])
    return out, bound, lse, e + 4 * U * np.maximum(np.abs(lse), 1)


def backward_want(part, io, scale, window=0, prefix=0):
    """((dq, bound), (dk, bound), (dv, bound)) of one sequence."""
    q, k, v, do = part
    Hh, n, d = q.shape
    h = H16 if io == "bf16" else 0.0
    got = ao.attention_backward(q, k, v, do, scale, window, prefix)
    out, ob, lse, lb = forward_want(part, io, scale, window, prefix)
    e = _weight_error(q, k, n, scale) + lb.max(initial=0)
    _, _, nv, ndo = _norms(q, k, v, do)
    edp = 8 * U * np.sqrt(d) * nv * ndo
    bounds = [np.zeros_like(t) for t in (q, k, v)]
    mask = ao.seen(n, window, prefix)
    r = 4 * U * np.sqrt(max(n * Hh // k.shape[0], 1))
    for i in range(Hh):
        kh = i // (Hh // k.shape[0])
        P, _ = ao.weights(q[i], k[kh], mask, scale)
        dP = do[i] @ v[kh].T
        D = (do[i] * out[i]).sum(-1, keepdims=True)
        eD = edp + (np.abs(do[i]) * ob[i]).sum(-1, keepdims=True)
        dS = np.abs(P * (dP - D))
        edS = P * (edp + eD) + (e + h + r) * dS
        bounds[0][i] = scale * edS @ np.abs(k[kh])
        bounds[1][kh] += scale * edS.T @ np.abs(q[i])
        bounds[2][kh] += (e + h + r) * (P.T @ np.abs(do[i]))
    return [(g, b + (h + U) * np.abs(g)) for g, b in zip(got, bounds)]


def near(name, got, want, bound):
    got = got.double().cpu().numpy() if hasattr(got, "cpu") else got
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert np.isfinite(got).all(), name
    off = np.abs(got - want) / np.maximum(bound, 1e-300)
    worst = off.max(initial=0)
    assert worst <= 1, f"{name}: {worst:.2f} of the bound at {np.unravel_index(off.argmax(), off.shape)}"
