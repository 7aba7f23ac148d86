"""Causal attention over prompts and its gradient against the fp64 oracle; bounds in attention_util.py."""
import numpy as np
import pytest

from attention_util import backward_want, dtype, forward_want, make, near, packed, padded

pytestmark = pytest.mark.gpu

#          H  Hk  sizes                      d   io    window prefix
CASES = [(1, 1, [1], 64, "bf16", 0, 0),
         (2, 1, [1, 2, 3], 16, "f32", 0, 0),
         (3, 3, [7], 1, "f32", 0, 0),
         (2, 2, [33, 31], 33, "bf16", 0, 0),
         (2, 2, [65, 0, 64], 48, "f32", 0, 0),
         (4, 2, [127, 129, 128], 64, "bf16", 0, 0),
         (4, 1, [200, 5], 128, "bf16", 0, 0),
         (6, 2, [150], 127, "f32", 0, 0),
         (6, 2, [131, 70], 96, "bf16", 0, 0),
         (2, 2, [140], 100, "bf16", 0, 0),
         (2, 2, [300], 128, "f32", 0, 0),
         (8, 8, [520], 64, "bf16", 0, 0),
         (2, 1, [260], 64, "bf16", 1, 0),
         (2, 1, [260], 32, "f32", 1, 1),
         (2, 2, [400, 37], 64, "bf16", 30, 0),
         (2, 2, [400], 80, "f32", 100, 7),
         (4, 2, [700], 64, "bf16", 129, 70),
         (2, 2, [333], 40, "bf16", 64, 64),
         (2, 2, [100], 64, "bf16", 1000, 3),
         (2, 2, [100], 64, "f32", 3, 1000),
         (1, 1, [1100], 72, "bf16", 257, 200)]


def _masked(t, parts, width):
    """Rows of [B, .., N, ..] past the lengths, as a list of views (dim 2 of 4, or 1 of 3)."""
    return [t[b, :, p[0].shape[1]:] if t.dim() == 4 else t[b, p[0].shape[1]:] for b, p in enumerate(parts)]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_padded(case):
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    H, Hk, sizes, d, io, window, prefix = case
    N = max(max(sizes), 1) + 3
    parts = make(1, H, Hk, sizes, d, io)
    nan = float("nan")
    q, k, v, do = (padded(parts, i, N, io, nan) for i in range(4))   # nothing past a length is read
    do = do.transpose(1, 2).reshape(len(sizes), N, H * d).contiguous()
    n = torch.tensor(sizes, dtype=torch.int32, device="cuda")
    kw = dict(lengths=n, window=window, prefix=prefix)
    out = torch.full((len(sizes), N, H * d), 3.0, dtype=dtype(io), device="cuda")
    lse = torch.full((len(sizes), H, N), 4.0, device="cuda")
    got = tmm.attention(q, k, v, out=out, lse_out=lse, **kw)
    assert got[0] is out and got[1] is lse
    grad = tmm.attention_backward(q, k, v, out, lse, do, **kw)
    scale = d ** -0.5
    for b, p in enumerate(parts):
        m = sizes[b]
        assert (out[b, m:] == 3).all() and (lse[b, :, m:] == 4).all()
        for name in ("q", "k", "v"):
            assert (grad[name][b, :, m:] == 0).all()
        if not m:
            continue
        o, ob, l, lb = forward_want(p, io, scale, window, prefix)
        near("out", out[b, :m].reshape(m, H, d).transpose(0, 1), o, ob)
        near("lse", lse[b, :, :m], l, lb)
        for name, (w, wb) in zip("qkv", backward_want(p, io, scale, window, prefix)):
            near("d" + name, grad[name][b, :, :m], w, wb)
    new = tmm.attention(q, k, v, **kw)
    for b, m in enumerate(sizes):
        assert torch.equal(new[0][b, :m], out[b, :m]) and (new[0][b, m:] == 0).all() and (new[1][b, :, m:] == 0).all()


@pytest.mark.parametrize("case", CASES, ids=str)
def test_packed(case):
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    H, Hk, sizes, d, io, window, prefix = case
    sizes = [0] + sizes + [1, 0, 40]
    first, total = 5, 5 + sum(sizes) + 4          # rows before the first sequence and behind the last
    parts = make(2, H, Hk, sizes, d, io)
    nan = float("nan")
    q, k, v, do = (packed(parts, i, total, first, io, nan) for i in range(4))
    do = do.reshape(total, H * d)
    at = np.concatenate([[first], first + np.cumsum(sizes)])
    kw = dict(offsets=torch.tensor(at, dtype=torch.int32, device="cuda"), window=window, prefix=prefix, scale=0.2)
    out = torch.full((total, H * d), 3.0, dtype=dtype(io), device="cuda")
    lse = torch.full((H, total), 4.0, device="cuda")
    tmm.attention(q, k, v, out=out, lse_out=lse, **kw)
    grad = tmm.attention_backward(q, k, v, out, lse, do, **kw)
    outside = torch.ones(total, dtype=torch.bool, device="cuda")
    outside[first:at[-1]] = False
    assert (out[outside] == 3).all() and (lse[:, outside] == 4).all()
    for name in ("q", "k", "v"):
        assert (grad[name][outside] == 0).all()
    for s, p in enumerate(parts):
        a, b = int(at[s]), int(at[s + 1])
        if a == b:
            continue
        o, ob, l, lb = forward_want(p, io, 0.2, window, prefix)
        near("out", out[a:b].reshape(b - a, H, d).transpose(0, 1), o, ob)
        near("lse", lse[:, a:b], l, lb)
        for name, (w, wb) in zip("qkv", backward_want(p, io, 0.2, window, prefix)):
            near("d" + name, grad[name][a:b].transpose(0, 1), w, wb)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_scores_far_apart(io):
    """Scores of hundreds: the running maximum moves often, weights of 0 and 1, nothing overflows."""
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    rng = np.random.default_rng(5)
    t = [torch.from_numpy(x).to(dtype(io)).cuda() for x in (40 * rng.standard_normal((1, 2, 300, 64)),
         rng.standard_normal((1, 2, 300, 64)), rng.standard_normal((1, 2, 300, 64)))]
    t[1][:, :, 100:200] *= 40
    p = tuple(x[0].double().cpu().numpy() for x in t)
    out, lse = tmm.attention(*t)
    o, ob, l, lb = forward_want(p, io, 0.125)
    near("out", out[0].reshape(300, 2, 64).transpose(0, 1), o, ob)
    near("lse", lse[0], l, lb)


def test_a_nan_stays_near_its_token():
    """Values: the queries from the token on, and at most 127 before it.  Keys: the queries that see it."""
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    for io in ("bf16", "f32"):
        q, k, v = (torch.randn(1, 2, 900, 64, device="cuda").to(dtype(io)) for _ in range(3))
        want = tmm.attention(q, k, v, window=200)[0]
        for bad in (float("nan"), float("inf")):
            w = v.clone()
            w[0, 1, 400, 3] = bad
            got = tmm.attention(q, k, w, window=200)[0]
            assert torch.equal(got[0, :400 - 127], want[0, :400 - 127]) and torch.equal(got[0, 727:], want[0, 727:])
            assert torch.equal(got[..., :64], want[..., :64])                  # the other head
            assert not torch.isfinite(got[0, 400:600, 64 + 3]).any()
        w = k.clone()
        w[0, 1, 400, 3] = float("nan")
        got = tmm.attention(q, w, v, window=200)[0]
        assert torch.equal(got[0, :400], want[0, :400]) and torch.equal(got[0, 600:], want[0, 600:])
        assert torch.isnan(got[0, 400:600, 64:]).all()


def test_offsets_that_are_not_in_order_or_in_range_stay_in_bounds():
    """Nothing is promised about the values; sequences in their place are right, and no other memory is touched."""
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    H, d, total = 2, 64, 300
    buf = torch.full((3 * total, H * d), 7.0, device="cuda", dtype=torch.bfloat16)
    q, k, v = (torch.randn(total, H, d, device="cuda").bfloat16() for _ in range(3))
    out, lse = buf[total:2 * total], torch.zeros(H, total, device="cuda")
    for cut in ([0, 100, 5000], [-50, 100, 200], [0, 250, 100, 300], [200, 100, 0], [400, 500, 600], [-5, -4, -3]):
        off = torch.tensor(cut, dtype=torch.int32, device="cuda")
        tmm.attention(q, k, v, offsets=off, out=out, lse_out=lse)
        g = tmm.attention_backward(q, k, v, out, lse, out, offsets=off)
        torch.cuda.synchronize()
        assert (buf[:total] == 7).all() and (buf[2 * total:] == 7).all() and g["q"].shape == q.shape
    off = torch.tensor([0, 100, 5000], dtype=torch.int32, device="cuda")
    got = tmm.attention(q, k, v, offsets=off)[0]
    want = tmm.attention(q, k, v, offsets=torch.tensor([0, 100, total], dtype=torch.int32, device="cuda"))[0]
    assert torch.equal(got, want)


def test_many_sequences_and_lengths_out_of_range():
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    rng = np.random.default_rng(6)
    sizes = rng.integers(0, 4, 5000)                       # more sequences than lanes, twice over
    at = np.concatenate([[0], np.cumsum(sizes)])
    total = int(at[-1])
    q, k, v = (torch.randn(total, 2, 32, device="cuda").bfloat16() for _ in range(3))
    out = tmm.attention(q, k, v, offsets=torch.tensor(at, dtype=torch.int32, device="cuda"))[0]
    want = torch.zeros(total, 2, 32, device="cuda")
    s = torch.from_numpy(np.repeat(np.arange(5000), sizes)).cuda()
    for back in range(4):                                  # scores with the tokens 0..3 before, where they are of the sequence
        pass
    x = torch.full((total, 2, 4), -float("inf"), device="cuda")
    for back in range(4):
        ok = torch.zeros(total, dtype=torch.bool, device="cuda")
        ok[back:] = s[back:] == s[:total - back]
        y = torch.zeros(total, 2, device="cuda")
        y[back:] = (q[back:].float() * k[:total - back].float()).sum(-1) * 32 ** -0.5
        x[..., back] = torch.where(ok[:, None], y, x[..., back])
    w = torch.softmax(x, -1)
    for back in range(4):
        want[back:] += w[back:, :, back, None] * v[:total - back].float()
    assert (out.reshape(total, 2, 32).float() - want).abs().max() <= 2 * 2 ** -8 * 6      # |v| < 6, two roundings
    q = torch.randn(2, 2, 50, 32, device="cuda")
    a = tmm.attention(q, q, q, lengths=torch.tensor([-3, 99], dtype=torch.int32, device="cuda"))
    b = tmm.attention(q, q, q, lengths=torch.tensor([0, 50], dtype=torch.int32, device="cuda"))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_gradient_adds_over_shared_heads_and_parts():
    """Few tiles of keys: their queries are shared by workgroups; many: by none.  The same sums either way."""
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, k, v = r(1, 8, 600, 64), r(1, 2, 600, 64), r(1, 2, 600, 64)
    do = r(1, 600, 512)
    few = tmm.attention_backward(q, k, v, *tmm.attention(q, k, v), do)
    B = 80                                                    # 80 x 2 x 5 tiles
    many_in = [t.repeat(B, 1, 1, 1) for t in (q, k, v)]
    many = tmm.attention_backward(*many_in, *tmm.attention(*many_in), do.repeat(B, 1, 1))
    for name in ("q", "k", "v"):
        assert torch.equal(many[name][0], many[name][B - 1])
        e = (few[name].float() - many[name][:1].float()).norm() / many[name][:1].float().norm()
        assert e <= 2 ** -8, name
    again = tmm.attention_backward(q, k, v, *tmm.attention(q, k, v), do)
    assert all(torch.equal(few[n], again[n]) for n in "qkv")


def test_empty_streams_and_graphs():
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    e = torch.empty(2, 4, 0, 64, device="cuda")
    out, lse = tmm.attention(e, e, e)
    assert out.shape == (2, 0, 256) and lse.shape == (2, 4, 0)
    g = tmm.attention_backward(e, e, e, out, lse, out)
    assert g["q"].shape == e.shape
    one = torch.randn(1, 2, 1, 64, device="cuda")
    # out = p v / l with l = p, whatever p rounds to: the planes of p and v leave out 4 u of p v, 1 / l and the last
    # product are a rounding each (the division a few units): 8 u |v|
    off = (tmm.attention(one, one, one)[0].reshape(2, 64) - one[0, :, 0]).abs()
    assert (off <= 8 * 2.0 ** -24 * one[0, :, 0].abs()).all()
    t = [torch.randn(2, 4, 300, 64, device="cuda").bfloat16() for _ in range(3)]
    do = torch.randn(2, 300, 256, device="cuda").bfloat16()

    def run():
        o, l = tmm.attention(*t, window=100, prefix=4)
        g = tmm.attention_backward(*t, o, l, do, window=100, prefix=4)
        return [o, l, g["q"], g["k"], g["v"]]

    want = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for turn in range(3):
        t[0].copy_(torch.randn_like(t[0]))
        graph.replay()
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), turn


def test_offsets_past_32_bits():
    """A packed row of more than 2^31 elements of q and of out: its last sequence is right."""
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    H, d = 16, 128
    total = (1 << 20) + 77
    q = torch.zeros(total, H, d, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.zeros(total, 1, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    parts = make(7, H, 1, [70], d, "bf16")
    for t, i in ((q, 0), (k, 1), (v, 2)):
        t[total - 70:] = packed(parts, i, 70, 0, "bf16")
    off = torch.tensor([0, 40, total - 70, total], dtype=torch.int32, device="cuda")
    off[2] = total - 70
    cut = torch.tensor([total - 200, total - 70, total], dtype=torch.int32, device="cuda")
    out, lse = tmm.attention(q, k, v, offsets=cut)
    o, ob, l, lb = forward_want(parts[0], "bf16", d ** -0.5)
    near("out", out[total - 70:].reshape(70, H, d).transpose(0, 1), o, ob)
    near("lse", lse[:, total - 70:], l, lb)
