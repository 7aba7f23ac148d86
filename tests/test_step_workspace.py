"""Host-only: the step's workspace has room for the parts' outputs up to a 16-byte border and their maxima and sums behind it."""
import pytest

from test_learned_neural_amd import titans_mem as tmm


@pytest.mark.parametrize("B,H,n,C,d", [(1, 1, 1, 800, 33), (1, 1, 1, 800, 32), (1, 3, 1, 5000, 1), (3, 1, 5, 900, 7)])
def test_pairs_start_at_16_bytes(B, H, n, C, d):
    got = tmm.attention_step_workspace_bytes(tmm.make_attention_step_desc(B, H, H, n, C, d))
    fits = [p for p in range(2, 65) if (B * H * n * p * d * 4 + 15) // 16 * 16 + B * H * n * p * 8 == got]
    assert len(fits) == 1 and got % 8 == 0, (got, fits)
