"""The delta memory's operators together, as a block runs them: input side ->
delta memory -> gated group norm, its gradient back through both, and a prompt
followed by single tokens in place.

Tolerances: every stage's oracle starts from the values that the GPU stage
before it left, so a stage answers for its own error alone (delta_util.py, and
the group norm's bound of half a bf16 step plus 64 fp32 units).
"""
import numpy as np
import pytest

from delta_util import U16, U32, check, tol32
from oracle import delta_oracle as do

pytestmark = pytest.mark.gpu


def _setup(seed, B, N, D, H, d):
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    x = r(B, N, D).bfloat16()
    k, v, q, alpha, eta, theta = tmm.input_side(
        x, (r(3, H * d, D) / D ** 0.5).bfloat16(), r(3, H * d, 4) / 2, (r(3, H, D) / D ** 0.5).bfloat16(), 0.5 * r(3, H),
        (0.1, 1.0, 1.0), H=H, d=d)
    W = r(B, H, d, d) / d ** 0.5
    return (k, v, q, alpha, theta, W), r(B, N, H * d).bfloat16(), 1 + 0.2 * r(H * d), 0.2 * r(H * d)


def _f64(*ts):
    return [t.double().cpu().numpy() for t in ts]


def test_block_forward_and_gradient():
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    B, N, D, H, d = 2, 150, 256, 4, 64
    mem, gate, weight, bias = _setup(41, B, N, D, H, d)
    n = torch.tensor([150, 97], dtype=torch.int32, device="cuda")
    live = np.arange(N)[None] < n.cpu().numpy()[:, None]
    y, W = tmm.delta_forward(*mem, lengths=n)
    out = tmm.group_norm(y, weight, bias, gate=gate, lengths=n)
    yr, Wr = do.delta_forward(*_f64(*mem), lengths=n.cpu().numpy())
    check("y", y, yr, "bf16", tol32(N, d))
    check("W", W, Wr, "f32", tol32(N, d))
    xs, z = _f64(y.transpose(1, 2), gate.reshape(B, N, H, d))
    w, b = (t.reshape(H, d) for t in _f64(weight, bias))
    ref = do.group_norm(xs, w, b, z) * live[..., None, None]
    got = out.double().cpu().numpy().reshape(ref.shape)
    assert np.all(np.abs(got - ref) <= U16 * np.abs(ref) + 64 * U32 * np.maximum(np.abs(ref), np.abs(z)))
    # and back
    gen = torch.Generator(device="cuda").manual_seed(42)
    dout = torch.randn(out.shape, generator=gen, device="cuda").bfloat16()
    dn = tmm.group_norm_backward(y, weight, bias, dout, gate=gate, lengths=n)
    dm = tmm.delta_backward(*mem, dy=dn["x"], lengths=n)
    want = do.delta_backward(*_f64(*mem), _f64(dn["x"])[0], lengths=n.cpu().numpy())
    for name in ("k", "v", "q", "alpha", "theta", "W_in"):
        check(name, dm[name], want[name], "bf16", 4 * tol32(N, d))
    dx, dz, dw, db = do.group_norm(xs, w, b, z, dout=_f64(dout)[0].reshape(ref.shape) * live[..., None, None])
    for name, a in (("x", dx.transpose(0, 2, 1, 3)), ("gate", dz.reshape(B, N, H * d))):
        a = a.reshape(dn[name].shape)
        check(name, dn[name].reshape(B, 1, -1), a.reshape(B, 1, -1), "bf16", 64 * U32)
    for name, a in (("weight", dw), ("bias", db)):
        e = dn[name].double().cpu().numpy() - a.sum((0, 1)).reshape(-1)
        assert np.all(np.abs(e) <= 64 * U32 * (2 * np.sqrt((a ** 2).sum((0, 1))).reshape(-1) + 2 * np.abs(a).max()))


def test_prompt_then_single_tokens_in_a_replayed_graph():
    """A prompt, then tokens one by one: the state in place, the step and its norm captured once and replayed."""
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    B, N, D, H, d, prompt = 3, 60, 128, 2, 64, 47
    mem, gate, weight, bias = _setup(43, B, N, D, H, d)
    k, v, q, alpha, theta, W0 = mem
    yr, Wr = do.delta_forward(*_f64(*mem))
    cut = lambda t, a, b: t[:, :, a:b].contiguous()
    state = W0.clone()
    tmm.delta_forward(*(cut(t, 0, prompt) for t in mem[:5]), state, W_out=state)
    step = [cut(t, 0, 1) for t in mem[:5]]
    z = gate[:, :1].contiguous()
    y = torch.empty_like(step[1])
    o = torch.empty_like(z)

    def one():
        tmm.delta_forward(*step, state, y_out=y, W_out=state)
        tmm.group_norm(y, weight, bias, gate=z, out=o)

    before = state.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        one()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    state.copy_(before)
    ys, os_ = [], []
    for t in range(prompt, N):
        for a, b in zip(step, mem[:5]):
            a.copy_(b[:, :, t:t + 1])
        z.copy_(gate[:, t:t + 1])
        graph.replay()
        ys.append(y.clone())
        os_.append(o.clone())
    check("y", torch.cat(ys, 2), yr[:, :, prompt:], "bf16", tol32(N, d))
    check("W", state, Wr, "f32", tol32(N, d))
    out = tmm.group_norm(torch.cat(ys, 2), weight, bias, gate=gate[:, prompt:].contiguous())
    assert torch.equal(out, torch.cat(os_, 1))
