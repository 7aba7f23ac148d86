"""Calls that are cut into segments: sequences that end before the last one."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
N = 60000     # 2 streams of 60000 tokens: 125 segments of 15 chunks


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
