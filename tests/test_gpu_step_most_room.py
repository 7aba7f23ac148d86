"""The step at the largest room of a cache, its places next to 2^31."""
import numpy as np
import pytest

from attention_util import H16, U, _weight_error, make, near
from oracle import attention_oracle as ao

pytestmark = pytest.mark.gpu


def test_most_room():
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    room, live = (1 << 31) - 32, 200
    part = make(81, 2, 1, [live], 1, "bf16")[0]
    q, k, v = (torch.from_numpy(x).bfloat16().cuda() for x in part[:3])
    kc, vc = (torch.zeros(1, 1, room, 1, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    kc[0, :, room - live:room - 2], vc[0, :, room - live:room - 2] = k[:, :-2], v[:, :-2]
    out = tmm.attention_step(q[None, :, -2:].contiguous(), kc, vc, torch.tensor([room], dtype=torch.int32, device="cuda"),
                             k_new=k[None, :, -2:].clone(), v_new=v[None, :, -2:].clone(), window=150)
    assert torch.equal(kc[0, :, room - live:], k) and torch.equal(vc[0, :, room - live:], v)
    f = [x[:, -151:] for x in part[1:3]]       # all that the two new tokens see
    want = ao.attention_step(part[0][:, -2:], *f, 1.0, window=150)
    size = ao.attention_step(part[0][:, -2:], f[0], np.abs(f[1]), 1.0, window=150)
    e = _weight_error(part[0], f[0], 151, 1.0)
    near("out", out.reshape(2, 2, 1).transpose(0, 1), want, (2 * e + H16) * size + (H16 + U) * np.abs(want))
