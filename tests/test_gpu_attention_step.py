"""Single tokens over a cache against the fp64 oracle; bounds in attention_util.py."""
import numpy as np
import pytest

from attention_util import H16, U, _weight_error, dtype, make, near, rounded
from oracle import attention_oracle as ao

pytestmark = pytest.mark.gpu

#          H  Hk n  room  lengths             d   io    window prefix
CASES = [(1, 1, 1, 1, [1, 0], 64, "bf16", 0, 0),
         (4, 2, 1, 40, [40, 1, 0, 33], 64, "bf16", 0, 0),
         (4, 2, 1, 40, [40, 1, 0, 32], 64, "f32", 0, 0),
         (6, 1, 3, 70, [70, 2, 0, 65, 3], 33, "bf16", 0, 0),
         (6, 1, 7, 300, [300, 5, 128], 48, "f32", 0, 0),     # 42 rows of a key head
         (16, 1, 5, 200, [200, 4, 129], 128, "bf16", 0, 0),  # 80 rows
         (2, 2, 2, 2000, [2000, 700], 96, "bf16", 0, 0),
         (2, 2, 1, 5000, [5000, 4097, 3], 128, "f32", 0, 0),
         (2, 2, 1, 5000, [5000, 4097, 3], 128, "bf16", 0, 0),
         (4, 4, 2, 3001, [3001, 1500], 1, "f32", 0, 0),
         (2, 1, 1, 900, [900, 100, 31], 64, "bf16", 1, 0),
         (2, 1, 2, 900, [900, 100, 31], 64, "f32", 65, 0),
         (2, 2, 3, 4000, [4000, 2222, 120], 80, "bf16", 500, 40),
         (2, 2, 1, 100, [100, 64], 100, "bf16", 1000, 1000)]


@pytest.mark.parametrize("stored", [False, True])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_step(case, stored):
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    H, Hk, n, room, lengths, d, io, window, prefix = case
    parts = make(11, H, Hk, [room] * len(lengths), d, io)
    rng = np.random.default_rng(12)
    nan, B = float("nan"), len(lengths)
    cache = torch.full((2, B, Hk, room, d), nan, dtype=dtype(io))
    new = torch.full((2, B, Hk, n, d), nan, dtype=dtype(io))
    q, qd = rounded(rng.standard_normal((B, H, n, d)), io)
    want, bound, after = np.zeros((B, n, H, d)), np.zeros((B, n, H, d)), None
    for b, m in enumerate(lengths):
        live = min(n, m)
        for i in range(2):
            t = torch.from_numpy(parts[b][1 + i][:, :m]).to(dtype(io))
            cache[i, b, :, :m] = t
            new[i, b, :, n - live:] = t[:, m - live:]
        k, v = (x[:, :m] for x in parts[b][1:3])
        want[b] = ao.attention_step(qd[b], k, v, d ** -0.5, window, prefix).transpose(1, 0, 2)
        if live:
            e, h = _weight_error(qd[b], k, m, d ** -0.5), H16 if io == "bf16" else 0.0
            size = ao.attention_step(qd[b], k, np.abs(v), d ** -0.5, window, prefix).transpose(1, 0, 2)
            bound[b] = (2 * e + h) * size + (h + U) * np.abs(want[b])
    after = cache.clone()
    if not stored:
        for b, m in enumerate(lengths):
            cache[:, b, :, max(m - n, 0):m] = nan
    k, v = (c.clone() for c in cache.cuda())
    kw = {} if stored else dict(k_new=new[0].cuda(), v_new=new[1].cuda())
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out = torch.full((B, n, H * d), 5.0, dtype=dtype(io), device="cuda")
    assert tmm.attention_step(q.cuda(), k, v, ln, window=window, prefix=prefix, out=out, **kw) is out
    near("out", out.reshape(B, n, H, d), want, bound + 1e-30)
    for a, b in ((k, after[0]), (v, after[1])):       # the new rows in their places, nothing else written
        assert torch.equal(torch.nan_to_num(a.cpu().float(), 9.0), torch.nan_to_num(b.float(), 9.0))


def test_prompt_then_tokens_agree_with_the_whole():
    """The prompt's kernel over everything, and tokens one by one over the cache they fill: a captured, replayed step."""
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    B, H, Hk, N, d, start = 3, 4, 2, 300, 64, 250
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn(B, H, N, d, generator=g, device="cuda")
    k, v = (torch.randn(B, Hk, N, d, generator=g, device="cuda") for _ in range(2))
    kw = dict(window=90, prefix=3)
    whole = tmm.attention(q, k, v, **kw)[0]
    room = 320
    kc, vc = (torch.zeros(B, Hk, room, d, device="cuda") for _ in range(2))
    kc[:, :, :start], vc[:, :, :start] = k[:, :, :start], v[:, :, :start]
    ln = torch.full((B,), start, dtype=torch.int32, device="cuda")
    one = [t[:, :, :1].contiguous() for t in (q, k, v)]

    def step():
        ln.add_(1)
        return tmm.attention_step(one[0], kc, vc, ln, k_new=one[1], v_new=one[2], **kw)

    keep = [t.clone() for t in (ln, kc, vc)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for a, b in zip((ln, kc, vc), keep):
        a.copy_(b)
    for t in range(start, N):
        for a, b in zip(one, (q, k, v)):
            a.copy_(b[:, :, t:t + 1])
        graph.replay()
        # two fp32 sums over the same weights in another order
        assert (out[:, 0] - whole[:, t]).abs().max() <= 64 * U * 5, t
    assert torch.equal(kc[:, :, :N], k) and torch.equal(vc[:, :, :N], v) and (kc[:, :, N:] == 0).all()
    assert (ln == N).all()


def test_lengths_out_of_range_and_nothing_to_do():
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    q, k, v = (torch.randn(2, 2, n, 32, device="cuda") for n in (1, 20, 20))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    assert torch.equal(tmm.attention_step(q, k, v, i32(-7, 99)), tmm.attention_step(q, k, v, i32(0, 20)))
    assert tmm.attention_step(q[:, :, :0].contiguous(), k, v, i32(3, 4)).shape == (2, 0, 64)


def test_a_cache_past_32_bits():
    """A cache of more than 2^31 elements a head: its last tokens, and the ones stored behind them."""
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    d, room = 128, (1 << 24) + 100
    k, v = (torch.zeros(1, 1, room, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    parts = make(13, 2, 1, [80], d, "bf16")
    for t, i in ((k, 1), (v, 2)):
        t[0, :, room - 80:] = torch.from_numpy(parts[0][i]).bfloat16().cuda()
    new = [t[:, :, room - 1:].clone() for t in (k, v)]
    k[0, 0, room - 1], v[0, 0, room - 1] = 0, 0
    q = torch.from_numpy(parts[0][0][None, :, 79:]).bfloat16().cuda().contiguous()
    out = tmm.attention_step(q, k, v, torch.tensor([room], dtype=torch.int32, device="cuda"), window=80, k_new=new[0],
                             v_new=new[1])
    qd, kd, vd = parts[0][0][:, 79:], parts[0][1], parts[0][2]
    want = ao.attention_step(qd, kd, vd, d ** -0.5)
    size = ao.attention_step(qd, kd, np.abs(vd), d ** -0.5)
    e = _weight_error(qd, kd, 80, d ** -0.5)
    near("out", out.reshape(1, 2, d).transpose(0, 1), want, (2 * e + H16) * size + (H16 + U) * np.abs(want))
    assert torch.equal(k[:, :, room - 1:], new[0]) and torch.equal(v[:, :, room - 1:], new[1])
