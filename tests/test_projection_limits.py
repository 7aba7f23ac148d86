"""Host-only: which sizes the projection's two calls take.  Addresses are never
dereferenced: a call that is taken is seen by the overlap that it has on purpose."""
import pytest

from test_learned_neural_amd import titans_mem as tmm

X, W, OUT = 0x700000000000, 0x710000000000, 0x720000000000


def forward(rows, K, O, io="bf16", act=tmm.ACT_NONE):
    """pre_out is out: TM_ERR_ALIAS if the sizes are taken."""
    return tmm.raw_projection(tmm.make_projection_desc(rows, K, O, io, act), X, W, 0, 0, OUT, OUT, 0)


def backward(rows, K, O, io="bf16", act=tmm.ACT_NONE):
    return tmm.projection_backward_workspace_bytes(tmm.make_projection_desc(rows, K, O, io, act))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("act", [tmm.ACT_NONE, tmm.ACT_SILU])
@pytest.mark.parametrize("rows", [1, 64, 65, 5000])
@pytest.mark.parametrize("K,O", [(8192, 65536), (8192, 128256), (65536, 8192), (16384, 262144)])
def test_large_weights_are_taken(rows, K, O, io, act):
    assert forward(rows, K, O, io, act) == tmm.ERR_ALIAS
    assert backward(rows, K, O, io, act) > 0


def test_the_forward_call_does_not_answer_for_the_gradient():
    """A weight of 2^38 numbers: its rows are read, but nothing launches over all of it; its gradient would."""
    assert forward(1, 1 << 19, 1 << 19) == tmm.ERR_ALIAS
    assert backward(1, 1 << 19, 1 << 19) == tmm.ERR_UNSUPPORTED
    # rows by K that dx has, and out does not
    assert forward(1 << 30, 1 << 15, 8, "f32") == tmm.ERR_ALIAS
    assert backward(1 << 30, 1 << 15, 8, "f32") == tmm.ERR_UNSUPPORTED


def test_too_many_channels_or_tiles():
    for K, O in (((1 << 22) + 1, 8), (8, (1 << 22) + 1)):
        assert forward(1, K, O) == tmm.ERR_UNSUPPORTED and backward(1, K, O) == tmm.ERR_UNSUPPORTED
    assert forward(1 << 40, 8, 8) == tmm.ERR_UNSUPPORTED and backward(1 << 40, 8, 8) == tmm.ERR_UNSUPPORTED
