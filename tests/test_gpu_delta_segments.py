"""Calls that are cut into segments, where a segment's map is not what a token
meets: growth that overflows over a segment and nowhere in the recurrence, and
sequences that end before the last segment."""
import numpy as np
import pytest

from delta_util import U32, check, tol32

pytestmark = pytest.mark.gpu
N, SEG = 60000, 480     # 2 streams of 60000 tokens: 125 segments of 15 chunks
GROWTH = -0.25          # 1.25^480 is 2^154; over 32 tokens it is 1262


def recurrence(k, v, q, alpha, theta, W):
    """fp64, one stream: y and W."""
    y = np.zeros_like(v)
    for t in range(len(k)):
        W = (1 - alpha[t]) * W
        W = W + theta[t] * np.outer(v[t] - W @ k[t], k[t])
        y[t] = W @ q[t]
    return y, W


def problem(d, used, io, alpha, seed=1):
    """Two streams whose keys replace column t mod used (theta = 1): no column that a key touches grows for more than
    `used` tokens."""
    import torch
    rng = np.random.default_rng([seed, d, used])
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    k = np.eye(d)[np.arange(N) % used][None, None].repeat(2, 1)
    q = np.where(np.arange(d) < used, rng.standard_normal((1, 2, N, d)), 0)
    t = {"k": torch.from_numpy(k).to(dt), "v": torch.from_numpy(rng.standard_normal((1, 2, N, d))).to(dt),
         "q": torch.from_numpy(q).to(dt), "alpha": torch.from_numpy(np.broadcast_to(alpha, (1, 2, N)).copy()).float(),
         "theta": torch.ones(1, 2, N), "W_in": torch.from_numpy(rng.standard_normal((1, 2, d, d))).float()}
    return t


def run(t, **kw):
    from test_learned_neural_amd import titans_mem as tmm
    B, H, _, d = t["v"].shape
    assert tmm.delta_workspace_bytes(tmm.make_delta_desc(B, H, t["k"].shape[1], N, d, "bf16" if t["k"].element_size() == 2 else "f32")) > 0
    return tmm.delta_forward(*(t[n].cuda() for n in ("k", "v", "q", "alpha", "theta", "W_in")), **kw)


def compare(t, y, W, io, d, used):
    """A column grows by 1.25 `used` times before it is replaced by v, in a chunk of 32 tokens 1 + 31 // used times.
    The chunk's form has every one of them as terms of its own: the column of its start grown past all replacements,
    and each residual grown past the later ones.  They are up to 1.25^(used (1 + 31 // used)) times what is left after
    the last replacement, and each is rounded less than 16 times (the decay's exponent and power, the products and
    their sums): 16 u of that factor, relative to the new column, beside what any recurrence of N tokens is off."""
    ref = [recurrence(*(t[n][0, h].double().numpy() for n in ("k", "v", "q", "alpha", "theta", "W_in"))) for h in range(2)]
    yr, Wr = (np.stack([r[i] for r in ref])[None] for i in range(2))
    assert np.abs(Wr).max() < 1e30
    tol = tol32(N, d) + 16 * U32 * (1 - GROWTH) ** (used * (1 + 31 // used))
    check("y", y, yr, io, tol)
    check("W", W, Wr, "f32", tol)


@pytest.mark.parametrize("d,io", [(40, "bf16"), (24, "f32"), (100, "f32")])
def test_growth_in_the_padding_of_a_width(d, io):
    """d is no multiple of 16: the rows that pad a map are no input of the memory."""
    used = min(d, 40)       # (d = 100: the other columns start at zero and stay so)
    t = problem(d, used, io, GROWTH)
    t["W_in"][..., used:] = 0
    y, W = run(t)
    compare(t, y, W, io, d, used)


@pytest.mark.parametrize("d,io", [(48, "bf16"), (64, "f32"), (128, "bf16")])
def test_growth_where_no_key_reaches(d, io):
    """A column that no key touches and that is zero stays zero, however far its map has grown."""
    t = problem(d, 40, io, GROWTH)
    t["W_in"][..., 40:] = 0
    y, W = run(t)
    assert (W[..., 40:] == 0).all()
    compare(t, y, W, io, d, 40)


@pytest.mark.parametrize("inplace", [False, True])
def test_growth_of_a_column_that_starts_small(inplace):
    """2^154 over one segment, from 1e-30: finite in the recurrence.  A second stream that only decays is unharmed."""
    d = 48
    alpha = np.full((1, 2, N), 0.01)
    alpha[0, 0, 21 * SEG:22 * SEG] = GROWTH
    alpha[:, :, :21 * SEG] = 0.0
    t = problem(d, 40, "f32", alpha)
    t["W_in"][..., 40:] *= 1e-30
    t["q"][:, :, 20 * SEG:, 44] = 1e-12
    if inplace:
        from test_learned_neural_amd import titans_mem as tmm
        g = {n: x.cuda() for n, x in t.items()}
        y, W = tmm.delta_forward(*(g[n] for n in ("k", "v", "q", "alpha", "theta", "W_in")), W_out=g["W_in"])
        assert W is g["W_in"]
    else:
        y, W = run(t)
    compare(t, y, W, "f32", d, 40)


def test_a_nan_in_a_late_segment_leaves_the_tokens_before_it():
    t = problem(64, 40, "bf16", 0.01)
    t["v"][0, 1, 30000, 3] = float("nan")
    y, W = run(t)
    t["v"][0, 1, 30000, 3] = 0
    want, _ = run(t)
    assert y[0, 1, 30000:, 3].isnan().any() and W[0, 1, 3].isnan().any()
    y[0, 1, 30000 // 32 * 32:, 3] = want[0, 1, 30000 // 32 * 32:, 3]
    e = (y.double() - want.double()).norm() / want.double().norm()
    assert float(e) <= 2 * (tol32(N, 64) + 2.0 ** -8), float(e)


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("d,io", [(64, "bf16"), (40, "f32")])
def test_a_state_without_tokens_is_copied_bit_by_bit(d, io, inplace):
    """W_out is W_in for length 0, infinities, NaN, zeros' signs and denormals among its values."""
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    g = {n: x.cuda() for n, x in problem(d, min(d, 40), io, 0.01).items()}
    two = {n: torch.cat([x, x]) for n, x in g.items()}
    odd = torch.tensor([float("inf"), float("-inf"), float("nan"), -0.0, 1e-42, -1e-40, 3e38], device="cuda")
    two["W_in"][1, 0, :7, 5] = odd
    two["W_in"][1, 1, 2, :7] = odd
    before = two["W_in"][1].clone()
    n = torch.tensor([N, 0], dtype=torch.int32, device="cuda")
    y, W = tmm.delta_forward(*(two[x] for x in ("k", "v", "q", "alpha", "theta", "W_in")), lengths=n,
                             W_out=two["W_in"] if inplace else None)
    assert torch.equal(W[1].view(torch.int32), before.view(torch.int32))
    assert torch.isfinite(W[0]).all() and (y[1] == 0).all()


def test_replays_with_and_without_growth():
    """Captured once, over lengths that end inside a segment: maps that overflow in one replay are of use in the next."""
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    names = ("k", "v", "q", "alpha", "theta", "W_in")
    x = {n: t.cuda() for n, t in problem(48, 40, "bf16", GROWTH).items()}
    x["W_in"][..., 40:] = 0
    lengths = torch.tensor([30011], dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    call = lambda: tmm.delta_forward(*(x[n] for n in names), lengths=lengths)
    call()
    with torch.cuda.graph(graph):
        y, W = call()
    for rep, (alpha, n) in enumerate(((GROWTH, 30011), (0.05, 30011), (GROWTH, N), (GROWTH, 100), (0.05, N))):
        x["alpha"].fill_(alpha)
        lengths.fill_(n)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = tmm.delta_forward(*(x[i] for i in names), lengths=lengths)
        assert torch.equal(y, want[0]) and torch.equal(W, want[1]), rep
        assert torch.isfinite(W).all() and torch.isfinite(y).all() and (y[:, :, n:] == 0).all(), rep
