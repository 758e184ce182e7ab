"""A workspace of beam_select that was made for some rows, vocabulary and candidates serves every call of no more of each."""
import pytest

import speculative_decoding_verification_74_gb300 as sv
from test_operator4_checks import L  # noqa: F401


@pytest.mark.parametrize("V,K", [(1, 1), (100, 128), (4097, 8), (32000, 4), (151936, 8), (1 << 18, 128)])
def test_sizes_grow_with_rows(L, V, K):  # noqa: F811
    sizes = [sv.sv_beam_workspace_size(rows, V, K) for rows in range(0, 2000)]
    assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_sizes_grow_with_vocabulary_and_candidates(L):  # noqa: F811
    for rows in (1, 7, 64, 300, 1000):
        sizes = [sv.sv_beam_workspace_size(rows, V, 8) for V in range(1, 1 << 18, 997)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:]))
        sizes = [sv.sv_beam_workspace_size(rows, 32000, K) for K in range(1, 129)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.gpu
def test_one_workspace_for_all_smaller_calls():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    x, scores = torch.randn((300, 60000), device="cuda"), -torch.rand((300, 1), device="cuda")
    ws = sv.beam_workspace(300, 60000, 8)
    for rows in (300, 299, 228, 152, 57, 14, 1):
        got = sv.beam_select(x[:rows], scores[:rows], 8, ws=ws)
        want = sv.beam_select(x[:rows], scores[:rows], 8)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
