"""Tree attention over a cache in 4 bits with a window and sinks, over pages of 64 slots and more: the window begins anywhere in a
page, and its first chunk does not follow the sinks' last one.  Batches large enough for a warp's part to hold both.  Bounds as
in test_gpu_attention4."""
import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv
from test_gpu_attention4 import case, check

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def lengths(page, window, n):
    """Lengths whose window begins at each chunk of 32 slots of a page, at its first, a middle and its last slot, pages further on."""
    each = [window - 1 + 2 * page + 32 * x + y for x in range(page // 32) for y in (0, 13, 31)]
    return (each * -(-n // len(each)))[:n]


# rows of a key/value head: 1, 4, 8 (tiles of 8 rows), 12 and 16 (of 16)
@pytest.mark.parametrize("page", [64, 128, 256])
@pytest.mark.parametrize("D,heads,kv_heads,tree", [(128, 32, 8, "one"), (128, 16, 16, "one"), (64, 64, 8, "one"), (64, 144, 12, "one"),
                                                   (128, 192, 12, "one"), (64, 12, 12, "wide"), (128, 12, 12, "mixed")])
def test_window_begins_within_a_page(page, D, heads, kv_heads, tree):
    for window, sinks in ((70, 4), (100, 40)):
        lens = lengths(page, window, 160)
        c = case(lens, [tree] * len(lens), heads, kv_heads, D, page, seed=page + window)
        ws = sv.attention_workspace(c["cache"], heads)
        check(c, window=window, sinks=sinks, ws=ws)
        assert sv.sv_query_status(ws) == (sv.SV_OK, 0)


@pytest.mark.parametrize("D,heads", [(64, 32), (128, 192)])
def test_a_missing_page_behind_the_sinks_is_reported(D, heads):
    page, window, sinks = 128, 70, 4
    lens = lengths(page, window, 160)
    c = case(lens, ["one"] * len(lens), heads, 12 if heads == 192 else 8, D, page, seed=1)
    ws = sv.attention_workspace(c["cache"], heads)
    want, want_lse = check(c, window=window, sinks=sinks, ws=ws)
    bad = list(range(0, len(lens), 5))
    for i in bad:
        c["cache"].page_table[i, (lens[i] - window + 1) // page] = -1
    out, lse = sv.tree_attention(c["q"], c["cache"], 0, c["lens"], c["offs"], c["parent"], c["nmax"], window=window, sinks=sinks, ws=ws)
    assert sv.sv_query_status(ws)[1] == sv.SV_DEV_BAD_PAGE
    for i in range(len(lens)):
        if i in bad:
            assert (out[i] == 0).all() and (lse[i] == -torch.inf).all()
        else:
            assert torch.equal(out[i], want[i]) and torch.equal(lse[i], want_lse[i])
