"""What the binding's entry points need is named with them."""
from io_aware_attention_flashattention_b200 import _lib, api

# reached through the scored and cache calls' own checks, not by name
HOST_ONLY = {"fa_score_span", "fa_cache4_row", "fa_status_string", "fa_forward_dropout_heads",
             "fa_backward_dropout_heads"}


def test_every_entry_point_and_its_workspace_size_is_named():
    assert set(_lib.SIGNATURES) - HOST_ONLY <= set(api.__all__)
    assert len(set(api.__all__)) == len(api.__all__)
    for name in api.__all__:
        assert hasattr(api, name)
