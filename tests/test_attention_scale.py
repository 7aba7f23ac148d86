"""Host-only: the scales that the attention's calls take.  scores go through base 2, where a scale above 2.3e38 is infinite."""
import pytest

from test_learned_neural_amd import titans_mem as tmm


@pytest.mark.parametrize("scale,taken", [(1e-45, True), (0.125, True), (2e38, True), (2.4e38, False), (3e38, False), (0.0, False)])
def test_scale(scale, taken):
    prompt = tmm.attention_backward_workspace_bytes(tmm.make_attention_desc(1, 1, 1, 5, 8, scale=scale))
    step = tmm.attention_step_workspace_bytes(tmm.make_attention_step_desc(1, 1, 1, 1, 8, 8, scale=scale))
    assert (prompt > 0 and step == 0) if taken else (prompt == step == tmm.ERR_INVALID)
