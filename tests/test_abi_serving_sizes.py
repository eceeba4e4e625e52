"""Sizes of the serving calls that an int does not hold are refused, not cut (CPU)."""
import pytest

from gqa_decode_attention_sm_gb300 import api
from gqa_decode_attention_sm_gb300 import build as gbuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32 + 8, -2 ** 32 + 8, 2 ** 64 + 1])
def test_sizes_past_an_int(big):
    for call in (lambda: api.evict_workspace_size(1, big), lambda: api.evict_workspace_size(big, 8),
                 lambda: api.weights_workspace_size(big, 64), lambda: api.weights_workspace_size(1, big),
                 lambda: api.weights_workspace_size(1, 64, big)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_sizes_are_whole_numbers():
    for bad in (8.0, "8", None):
        with pytest.raises(TypeError):
            api.evict_workspace_size(1, bad)
        with pytest.raises(TypeError):
            api.weights_workspace_size(1, bad)
    assert api.evict_workspace_size(1, 8) > 0
