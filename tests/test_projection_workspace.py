"""Host-only: what the projection's gradient asks for beside its results."""
import pytest

from test_learned_neural_amd import titans_mem as tmm


@pytest.mark.parametrize("rows,K,O", [(65536, 1024, 1024), (1001, 500, 777), (3, 5, 7), (0, 8, 8)])
def test_dz_is_kept_once_in_fp32_and_in_two_numbers_in_bf16(rows, K, O):
    ws = lambda io, act: tmm.projection_backward_workspace_bytes(tmm.make_projection_desc(rows, K, O, io, act))  # noqa: E731
    dz = (rows * O * 4 + 15) // 16 * 16
    assert ws("f32", tmm.ACT_SILU) - ws("f32", tmm.ACT_NONE) == dz
    # bf16: two planes, and at most one set of parts of the weight's gradient more
    two = 2 * ((rows * O * 2 + 15) // 16 * 16)
    more = ws("bf16", tmm.ACT_SILU) - ws("bf16", tmm.ACT_NONE) - two
    assert 0 <= more <= 128 * O * K * 4
