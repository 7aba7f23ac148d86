"""Steps whose parts hold odd counts of numbers: rows * parts * d that no 16 bytes divide."""
import numpy as np
import pytest

from attention_util import H16, U, _weight_error, dtype, make, near
from oracle import attention_oracle as ao

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,n,room,d,io", [(1, 1, 800, 33, "bf16"), (1, 1, 800, 33, "f32"), (1, 1, 800, 1, "f32"),
                                           (3, 1, 1900, 7, "bf16"), (1, 5, 1300, 127, "f32"), (1, 1, 17000, 9, "bf16")])
def test_step(H, n, room, d, io):
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    assert tmm.attention_step_workspace_bytes(tmm.make_attention_step_desc(1, H, H, n, room, d, io)) > 0   # several parts
    q, k, v, _ = make(21, H, H, [room], d, io)[0]
    q = q[:, :n]
    t = [torch.from_numpy(np.ascontiguousarray(x))[None].to(dtype(io)).cuda() for x in (q, k, v)]
    out = tmm.attention_step(*t, torch.tensor([room], dtype=torch.int32, device="cuda"))
    want, size = (ao.attention_step(q, k, x, d ** -0.5) for x in (v, np.abs(v)))
    e, h = _weight_error(q, k, room, d ** -0.5), H16 if io == "bf16" else 0.0
    near("out", out.reshape(n, H, d).transpose(0, 1), want, (2 * e + h) * size + (h + U) * np.abs(want))
