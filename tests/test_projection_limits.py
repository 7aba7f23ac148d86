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


@pytest.mark.parametrize("act", [tmm.ACT_NONE, tmm.ACT_SILU])
def test_small_fp32_tiles_have_1024_threads(act):
    """dx of fp32 rows that are not whole pieces goes by tiles of 64 x 64 and 1024 threads, 2^22 of which are
    2^32 threads, too many for a launch.  The forward call goes by 128 x 128 and 256 threads.  (Launches are
    rounded up to eight workgroups.)"""
    most = 64 * ((1 << 22) - 8)
    for K, O in ((3, 3), (64, 3), (3, 64), (1, 4)):
        assert backward(most, K, O, "f32", act) > 0
        assert backward(most + 1, K, O, "f32", act) == tmm.ERR_UNSUPPORTED
        assert backward(300_000_000, K, O, "f32", act) == tmm.ERR_UNSUPPORTED
        assert forward(300_000_000, K, O, "f32", act) == tmm.ERR_ALIAS
    # whole pieces: 128 x 128 by 256 threads
    assert backward(300_000_000, 4, 4, "f32", act) > 0 and backward(128 * ((1 << 24) - 8), 4, 4, "f32", act) > 0
    assert backward(128 * ((1 << 24) - 8) + 1, 4, 4, "f32", act) == tmm.ERR_UNSUPPORTED
    # bf16: small tiles of 256 threads
    assert backward(64 * ((1 << 24) - 8), 3, 3, "bf16", act) > 0
    assert backward(64 * ((1 << 24) - 8) + 1, 3, 3, "bf16", act) == tmm.ERR_UNSUPPORTED
    # large odd tiles forward
    assert forward(128 * ((1 << 24) - 8), 3, 3, "f32", act) == tmm.ERR_ALIAS
    assert forward(128 * ((1 << 24) - 8) + 1, 3, 3, "f32", act) == tmm.ERR_UNSUPPORTED
