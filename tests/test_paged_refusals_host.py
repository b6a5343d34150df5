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
