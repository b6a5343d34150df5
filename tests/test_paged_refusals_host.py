"""Refusals of the paged cache's calls that its other host test does not make, before any launch.  (No call of this file may
pass: it would be launched.)"""
import ctypes

import pytest
import torch

from sparse_long_context_gb300 import _lib as L
from sparse_long_context_gb300 import ops
from tests.test_paged_host import attend, cache, desc, error


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


def test_the_attends_limits(lib):
    size = lambda **kw: lib.sls_paged_decode_attend_workspace_size(ctypes.byref(desc(**kw)))  # noqa: E731
    rows = dict(batch=2048, num_q_heads=8, num_kv_heads=2)  # 4096 of them: Cap/16 + 1 below 2^18
    assert size(**rows, capacity=16 * 262142) > 0
    assert size(**rows, capacity=16 * 262143) == 0
    assert attend(lib, d=desc(**rows, capacity=16 * 262143), c=cache(table=1 << 40)) == L.SLS_EUNSUPPORTED  # a table of 2 GB
    one = dict(batch=1, num_q_heads=1, num_kv_heads=1)
    assert size(**one, capacity=1 << 30) > 0
    assert attend(lib, d=desc(**rows), stride=262145) == L.SLS_EOVERFLOW
    assert attend(lib, d=desc(**rows), stride=262144, fixed=262144, size=64) == L.SLS_EWORKSPACE  # the lists are taken
    assert attend(lib, d=desc(**rows, page_size=64), stride=65537) == L.SLS_EOVERFLOW
    assert attend(lib, d=desc(**one), stride=1 << 27) == L.SLS_EOVERFLOW
    assert attend(lib, d=desc(**one), stride=(1 << 27) - 1, fixed=0, size=64) == L.SLS_EWORKSPACE
