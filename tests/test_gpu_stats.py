"""sls_stats counts the attends over the 8-bit and the paged cache, and which way a paged selection went."""
import pytest
import torch

from sparse_long_context_gb300 import ops

pytestmark = pytest.mark.gpu


def test_cache_calls_are_counted():
    ops.get_stats(reset=True)
    desc = ops.make_desc(2, 4, 2, 64, 16, 256, torch.bfloat16)
    paged = ops.PagedCache.empty(desc, 40, summaries=True)
    kv = torch.randn((2, 100, 2, 64), device="cuda").to(torch.bfloat16)
    q = torch.randn((2, 4, 64), device="cuda").to(torch.bfloat16)
    ops.paged_append(desc, paged, kv, kv)
    ops.get_stats(reset=True)
    idx = ops.paged_select_pages(desc, paged, q, 3)
    ops.paged_decode_attend(desc, paged, q, page_idx=idx)
    ops.paged_decode_attend(desc, paged, q)
    cores = ops.make_desc(2, 4, 2, 64, 16, 256, torch.bfloat16, cuda_cores=True)
    assert torch.equal(idx, ops.paged_select_pages(cores, paged, q, 3))
    wide = ops.make_desc(2, 4, 2, 64, 16, 16 * 9000, torch.bfloat16)
    ops.paged_select_pages(wide, ops.PagedCache.empty(wide, 40, summaries=True), q, 3)
    cache = ops.Kv8Cache.empty(desc, "int8", 64)
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    ops.kv8_append(desc, cache, kv, kv, lens)
    ops.kv8_decode_attend(desc, cache, q, lens)
    got = ops.get_stats(reset=True)
    assert got["attend_paged"] == 2 and got["attend_kv8"] == 1
    assert got["select_pages"] == 3 and got["select_paged_one_launch"] == 1
    assert got["attend_tma"] == got["attend_mma"] == got["attend_cuda_cores"] == 0
    assert not any(ops.get_stats().values())
