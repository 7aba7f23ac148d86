"""Host-only: every operator of the binding is a name of the package, too."""
import pytest

import test_learned_neural_amd as pkg
from test_learned_neural_amd import titans_mem as tmm


@pytest.mark.parametrize("name", ["forward", "retrieve", "delta_forward", "delta_backward", "group_norm",
                                  "group_norm_backward", "attention", "attention_backward", "attention_step",
                                  "projection", "projection_backward"])
def test_operator(name):
    assert getattr(pkg, name) is getattr(tmm, name)
