"""Page lists without columns have no memory, and a call without lists is one over every page: such lists are refused."""
import pytest
import torch

from sparse_long_context_gb300 import _lib as L
from sparse_long_context_gb300 import ops

pytestmark = pytest.mark.gpu


def setup():
    gen = torch.Generator("cuda").manual_seed(0)
    desc = ops.make_desc(2, 4, 2, 64, 16, 256, torch.bfloat16)
    new = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    ctx = torch.tensor([200, 130], dtype=torch.int32, device="cuda")
    return desc, new(2, 4, 64), new(2, 2, 256, 64), new(2, 2, 256, 64), ctx


NONE = torch.empty((4, 0), dtype=torch.int32)


@pytest.mark.parametrize("how", ["attend", "combine", "recall", "refined"])
@pytest.mark.parametrize("count", [False, True])
def test_row_caches(how, count):
    desc, q, k, v, ctx = setup()
    idx = NONE.cuda()
    n = torch.zeros(4, dtype=torch.int32, device="cuda") if count else None
    call = {"attend": lambda i: ops.sparse_decode_attend(desc, q, k, v, i, ctx, 2, count=n),
            "combine": lambda i: ops.sparse_decode_attend_combine(desc, q, k, v, i, ctx, 2, count=n),
            "recall": lambda i: ops.selection_recall(desc, q, k, i, ctx, count=n),
            "refined": lambda i: ops.refined_decode_attend_combine(desc, q, k, v, None, None, None, i,
                                                                   torch.zeros(4, dtype=torch.int32, device="cuda"), ctx)}[how]
    with pytest.raises((ValueError, L.SlsError), match="page_idx|block_idx|entr"):
        call(idx)
    call(torch.full((4, 1), -1, dtype=torch.int32, device="cuda"))  # lists that hold nothing
    ops.pipeline_check()


def test_eight_bit_cache():
    desc, q, k, v, ctx = setup()
    cache = ops.Kv8Cache.empty(desc, "int8", 64)
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    ops.kv8_append(desc, cache, k.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous(), lens, new_len=ctx)
    with pytest.raises(ValueError, match="page_idx"):
        ops.kv8_decode_attend(desc, cache, q, lens, page_idx=NONE.cuda())
    out, lse = ops.kv8_decode_attend(desc, cache, q, lens, page_idx=torch.full((4, 1), -1, dtype=torch.int32, device="cuda"))
    assert not out.any() and bool((lse == -torch.inf).all())


def test_counts_without_lists_of_a_paged_cache():
    desc, q, k, v, ctx = setup()
    cache = ops.PagedCache.empty(desc, 40)
    ops.paged_append(desc, cache, k.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous(), new_len=ctx)
    count = torch.ones(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="count"):
        ops.paged_decode_attend(desc, cache, q, count=count)
    with pytest.raises(ValueError, match="k_fixed"):
        ops.paged_decode_attend(desc, cache, q, k_fixed=3)
    ops.paged_decode_attend(desc, cache, q)
    lists = torch.arange(3, dtype=torch.int32, device="cuda").repeat(4, 1)
    one = ops.paged_decode_attend(desc, cache, q, page_idx=lists, count=count)
    fixed = ops.paged_decode_attend(desc, cache, q, page_idx=lists, k_fixed=1)
    assert torch.equal(one[0], fixed[0]) and torch.equal(one[1], fixed[1])
    ops.pipeline_check()
