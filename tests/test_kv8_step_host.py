"""Refusals of the decode step over the 8-bit cache, before anything is allocated or appended."""
import pytest
import torch

from sparse_long_context_gb300 import ops


def make(page=16, cap=1024, flags=None, **kw):
    desc = ops.make_desc(2, 8, 2, 64, page, cap, torch.bfloat16, **(flags or {}))
    return ops.Kv8Decode(desc, ops.make_rope(8, 2, 64, torch.bfloat16), "int8", 64, device="cpu", **kw)


@pytest.mark.parametrize("kw,what", [
    (dict(page=8, k_budget=4), "pages of >= 16 tokens"), (dict(page=1, k_budget=4), "pages of >= 16 tokens"),
    (dict(k_budget=65), "k_budget"), (dict(k_budget=-1), "k_budget"), (dict(k_budget=4, n_sink_pages=5), "k_budget"),
    (dict(k_budget=4, n_sink_pages=-1), "k_budget"), (dict(k_budget=4, n_local_tokens=-16), "k_budget"),
    (dict(k_budget=4, n_sink_pages=1, n_local_tokens=33), "k_budget"), (dict(k_budget=4, mass=True), "weight sums"),
    (dict(flags=dict(cuda_cores=True)), "path flags"),
])
def test_step_refuses_what_its_first_call_would(kw, what):
    with pytest.raises(ValueError, match=what):
        make(**kw)


@pytest.mark.parametrize("kw", [dict(k_budget=64), dict(k_budget=4, n_sink_pages=1, n_local_tokens=32), dict(page=8)])
def test_step_takes_what_its_calls_take(kw):
    """(Without a GPU the cache's buffers are what is refused next.)"""
    with pytest.raises(ValueError, match="CUDA"):
        make(**kw)
