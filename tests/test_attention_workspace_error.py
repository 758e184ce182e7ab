"""A workspace size that cannot be given says why, not what an earlier call's error was."""
import pytest

import speculative_decoding_verification_74_gb300 as sv
from test_operator4_checks import FAKE, L, cache4  # noqa: F401


def cache16(**over):
    good = dict(k=FAKE, v=FAKE, layer_stride=8 * 16 * 128, page_stride=16 * 128, slot_stride=128, head_stride=64, layers=2, pages=8,
                page_size=16, kv_heads=2, head_dim=64, page_refs=FAKE)
    return sv.sv_cache(**{**good, **over})


@pytest.mark.parametrize("make,size", [(cache16, "sv_attention_workspace_size"), (cache4, "sv_attention4_workspace_size")])
@pytest.mark.parametrize("heads", [0, 3, 258])
def test_heads(L, make, size, heads):  # noqa: F811
    assert getattr(sv, size)(make(), 4) > 0
    assert getattr(sv, size)(make(layers=0), 4) == 0 and b"layers=0" in L.sv_last_error_string()
    assert getattr(sv, size)(make(), heads) == 0
    assert b"q_heads=%d" % heads in L.sv_last_error_string()
