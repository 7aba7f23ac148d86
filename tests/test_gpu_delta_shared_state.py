"""One state, in place, and two calls at once: the sequences without tokens in a call are another's."""
import pytest

pytestmark = pytest.mark.gpu
NAMES = ("k", "v", "q", "alpha", "theta")


def _problem(B, H, N, d, io):
    import torch
    g = torch.Generator(device="cuda").manual_seed(6)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    unit = lambda: torch.nn.functional.normalize(r(B, H, N, d), dim=-1).to(dt)
    return {"k": unit(), "v": r(B, H, N, d).to(dt), "q": unit(), "alpha": 0.1 * torch.rand(B, H, N, device="cuda"),
            "theta": torch.rand(B, H, N, device="cuda")}, r(B, H, d, d)


#         B   H   N     d    io      (single tokens, chunks, segments)
SHAPES = [(192, 16, 1, 128, "bf16"), (192, 16, 1, 128, "f32"), (64, 16, 2, 33, "bf16"), (64, 16, 40, 64, "bf16"),
          (32, 8, 70, 128, "f32"), (2, 2, 3000, 64, "bf16"), (4, 1, 3000, 100, "f32")]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_two_calls_share_a_state(shape):
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    B, H, N, d, io = shape
    x, W0 = _problem(*shape)
    even = torch.arange(B, device="cuda") % 2 == 0
    lengths = [torch.where(even == bool(i), 0, N).int() for i in range(2)]
    want, W = [], W0
    for n in lengths:       # one after the other, each into a new state
        y, W = tmm.delta_forward(*(x[n_] for n_ in NAMES), W, lengths=n)
        want.append(y)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = tmm.delta_workspace_bytes(tmm.make_delta_desc(B, H, H, N, d, io))
    for rep in range(8):
        state = W0.clone()
        outs = [torch.zeros_like(x["v"]) for _ in range(2)]
        scratch = [torch.empty(max(ws, 16), dtype=torch.uint8, device="cuda") for _ in range(2)]
        torch.cuda.synchronize()
        for s, n, y, w in zip(streams, lengths, outs, scratch):
            with torch.cuda.stream(s):
                tmm.delta_forward(*(x[n_] for n_ in NAMES), state, lengths=n, y_out=y, W_out=state, workspace=w)
        torch.cuda.synchronize()
        assert torch.equal(state, W), rep
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), rep


def test_a_slot_is_filled_while_others_step():
    """A new user's state comes into an idle slot by a copy on another stream."""
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    B, H, N, d = 192, 16, 1, 128
    x, W0 = _problem(B, H, N, d, "bf16")
    idle = B // 2
    n = (torch.arange(B, device="cuda") >= idle).int()
    _, W = tmm.delta_forward(*(x[n_] for n_ in NAMES), W0, lengths=n)
    side = torch.cuda.Stream()
    y = torch.zeros_like(x["v"])
    for rep in range(8):
        state, new = W0.clone(), W0[:idle] * (rep + 2)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            state[:idle].copy_(new)
        tmm.delta_forward(*(x[n_] for n_ in NAMES), state, lengths=n, y_out=y, W_out=state)
        torch.cuda.synchronize()
        assert torch.equal(state[:idle], new) and torch.equal(state[idle:], W[idle:]), rep
