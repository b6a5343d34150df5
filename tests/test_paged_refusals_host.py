"""Refusals of the paged cache's calls that its other host test does not make, before any launch.  (No call of this file may
pass: it would be launched.)"""
import ctypes

import pytest
import torch

from sparse_long_context_gb300 import _lib as L
from sparse_long_context_gb300 import ops
from tests.test_paged_host import attend, desc, error


def test_counts_without_lists(lib):
    assert attend(lib, idx=None) == L.SLS_EINVAL and "count" in error(lib)
    assert attend(lib, idx=None, stride=0, fixed=0) == L.SLS_EINVAL and "count" in error(lib)


def test_a_step_whose_rows_the_selection_does_not_take_is_refused_when_it_is_made():
    """262144 pages a row at most, where pages are selected; a device is not looked for before that."""
    def step(cap, **kw):
        d = ops.make_desc(2, 4, 2, 64, 16, cap, torch.bfloat16)
        return ops.PagedDecode(d, ops.make_rope(4, 2, 64, torch.bfloat16), 8, device="meta", **kw)
    with pytest.raises(ValueError, match="262144"):
        step(16 * 262145, k_budget=4)
    for cap, kw in ((16 * 262144, dict(k_budget=4)), (16 * 262145, {})):  # as far as the cache's tensors
        with pytest.raises(ValueError, match="CUDA tensor"):
            step(cap, **kw)
