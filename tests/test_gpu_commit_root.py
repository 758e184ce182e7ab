"""A commit whose tree's first node lies at a slot without a page (its reserve was refused, and the round went on): reported,
like every other node's."""
import os
import sys

import numpy as np
import pytest

import speculative_decoding_verification_74_gb300 as sv

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_cache import _gpu, i32, make, same  # noqa: E402, F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("accepted", [0, 1])
def test_a_first_node_without_a_page(accepted):
    cache, oracle = make(2, 3, 8, 2, 64, 2, 4)
    assert cache.reserve(i32([8, 6]), i32([3, 2])).tolist() == oracle.reserve([8, 6], [3, 2]).tolist() == [1, 1]
    cache.page_table[0, 1], cache.page_refs[oracle.table[0, 1]] = -1, 0
    oracle.refs[oracle.table[0, 1]] = 0
    oracle.table[0, 1] = -1
    path = np.asarray([[1, -1, -1], [1, -1, -1]])
    out = cache.commit(i32([8, 6]), i32([0, 3, 5]), i32(path), i32([accepted, 1]))
    assert out.tolist() == [9 + accepted, 8]
    assert sv.sv_query_status(cache.ws) == (sv.SV_ERR_DEVICE_INPUT, sv.SV_DEV_BAD_PAGE)
    same(cache, oracle)


def test_no_tree_or_a_refused_one_needs_no_page():
    cache, oracle = make(1, 3, 8, 2, 64, 3, 4)
    cache.reserve(i32([8, 8, 5]), i32([0, 0, 1]))
    oracle.reserve([8, 8, 5], [0, 0, 1])
    out = cache.commit(i32([8, 8, 5]), i32([0, 0, 2, 3]), i32([[-1, -1]] * 3), i32([0, -1, 0]))
    assert out.tolist() == [8, 8, 6]
    assert sv.sv_query_status(cache.ws) == (sv.SV_OK, 0)
    same(cache, oracle)
