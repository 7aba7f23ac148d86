"""Host-only: the rooms of a cache that the step takes."""
import pytest

from test_learned_neural_amd import titans_mem as tmm


@pytest.mark.parametrize("window", [0, 80])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_room(io, window):
    """Places are 32-bit: with more room the end of the last tile of 32 keys would not be one."""
    ok = lambda C: tmm.attention_step_workspace_bytes(  # noqa: E731
        tmm.make_attention_step_desc(1, 1, 1, 1, C, 1, io, window=window))
    assert ok((1 << 31) - 32) >= 0
    for C in ((1 << 31) - 31, (1 << 31) - 1):
        assert ok(C) == tmm.ERR_UNSUPPORTED, C


@pytest.mark.parametrize("B,H,Hk,n", [(1 << 20, 1 << 30, 1 << 19, 1 << 14), (1 << 24, 1, 1, 1), (1, 1, 1, 1 << 24),
                                      (1 << 22, 1 << 22, 1 << 22, 1 << 25)])
def test_too_many_queries(B, H, Hk, n):
    """2^24 and more, up to counts whose tiles pass 64 bits."""
    assert tmm.attention_step_workspace_bytes(tmm.make_attention_step_desc(B, H, Hk, n, 1, 1)) == tmm.ERR_UNSUPPORTED
