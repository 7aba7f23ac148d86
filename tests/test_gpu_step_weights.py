"""bf16 steps: the weights keep 16 bits where they meet the values, so that out is off by its own rounding.

u = 2^-24.  A weight is kept as what it is rounded to and what that rounding left,
each half a step of bf16 off at most: 2^-8 2^-9 of it (the remainder is half a step,
2^-8, of the weight at most, and is rounded by half a step of its own), taken as
2^-16.  With attention_util.py's e for the scores, the sums and their
rounding: out is off by (2 e + 2^-16) sum P |v| + (2^-8 + u) |out|."""
import numpy as np
import pytest

from attention_util import H16, U, _weight_error, make, near
from oracle import attention_oracle as ao

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,Hk,n,room,d,window,prefix", [
    (1, 1, 1, 40, 64, 0, 0), (4, 2, 1, 2000, 128, 0, 0), (8, 1, 3, 700, 33, 0, 0), (16, 1, 5, 300, 128, 0, 0),
    (2, 2, 2, 5000, 96, 0, 0), (4, 4, 1, 16384, 64, 0, 0), (2, 1, 1, 9000, 80, 300, 20), (2, 2, 1, 600, 16, 0, 0)])
def test_out_is_off_by_its_own_rounding(H, Hk, n, room, d, window, prefix):
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    q, k, v, _ = make(111, H, Hk, [room], d, "bf16")[0]
    q = q[:, :n]
    t = [torch.from_numpy(np.ascontiguousarray(x))[None].bfloat16().cuda() for x in (q, k, v)]
    out = tmm.attention_step(*t, torch.tensor([room], dtype=torch.int32, device="cuda"), window=window, prefix=prefix)
    want, size = (ao.attention_step(q, k, x, d ** -0.5, window, prefix) for x in (v, np.abs(v)))
    e = _weight_error(q, k, room, d ** -0.5)
    near("out", out.reshape(n, H, d).transpose(0, 1), want, (2 * e + 2.0 ** -16) * size + (H16 + U) * np.abs(want))
