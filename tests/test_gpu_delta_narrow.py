"""The delta memory's chunks, segments and gradient at widths of one tile or less."""
import pytest

from delta_util import check, cuda, make, tol32
from oracle import delta_oracle as do

pytestmark = pytest.mark.gpu
NAMES = ("k", "v", "q", "alpha", "theta", "W_in")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d", [1, 2, 3, 4, 5, 8, 12, 15, 16, 17, 20])
def test_chunks_and_gradient(d, io):
    from test_learned_neural_amd import titans_mem as tmm
    t, f = make(91, 2, 2, 1, 77, d, io, resets=True, lengths=[77, 40])
    g = cuda(t)
    a = [f[n] for n in NAMES]
    y, W = tmm.delta_forward(*(g[n] for n in NAMES), lengths=g["lengths"])
    yr, Wr = do.delta_forward(*a, f["lengths"])
    check("y", y, yr, io, tol32(77, d))
    check("W", W, Wr, "f32", tol32(77, d))
    got = tmm.delta_backward(*(g[n] for n in NAMES), dy=g["dy"], dW_out=g["dW"], lengths=g["lengths"])
    want = do.delta_backward(*a, f["dy"], f["dW"], f["lengths"])
    for name in NAMES:
        check(name, got[name], want[name], io, 4 * tol32(77, d))


@pytest.mark.parametrize("d,io", [(1, "f32"), (4, "bf16"), (8, "bf16"), (12, "f32"), (16, "bf16"), (17, "f32"), (20, "bf16")])
def test_segments(d, io):
    from test_learned_neural_amd import titans_mem as tmm
    N = 2500
    assert tmm.delta_workspace_bytes(tmm.make_delta_desc(1, 2, 1, N, d, io)) > 0
    t, f = make(92, 1, 2, 1, N, d, io, resets=True)
    g = cuda(t)
    y, W = tmm.delta_forward(*(g[n] for n in NAMES))
    yr, Wr = do.delta_forward(*(f[n] for n in NAMES))
    check("y", y, yr, io, tol32(N, d))
    check("W", W, Wr, "f32", tol32(N, d))
