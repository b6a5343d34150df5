"""The planted wait of the 8-bit attend's test hook is that of the first CTA with tokens, wherever the empty rows are."""
import numpy as np
import pytest
import torch

from sparse_long_context_gb300 import _lib as L
from sparse_long_context_gb300 import ops

pytestmark = pytest.mark.gpu


# the first rows empty: in clusters (a row's own is empty), in ranges (a first range that holds a row's start only)
@pytest.mark.parametrize("cap,lens", [(4096, [0, 200, 130]), (4096, [0, 0, 0, 4000]), (1 << 20, [0, 200, 130]),
                                      (1 << 17, [0] + [88] * 99), (1 << 17, [0] * 60 + [1504] + [88] * 99)])
def test_wait_that_gives_up_is_that_of_the_first_tokens(cap, lens):
    rng = np.random.default_rng(1)
    batch = len(lens)
    mk = lambda **kw: ops.make_desc(batch, 2, 1, 64, 16, cap, torch.bfloat16, **kw)  # noqa: E731
    desc = mk()
    cache = ops.Kv8Cache.empty(desc, "int8", 64)
    ctx = torch.zeros(batch, dtype=torch.int32, device="cuda")
    x = torch.from_numpy(rng.standard_normal((batch, max(lens), 2, 64))).to(torch.bfloat16).cuda()
    ops.kv8_append(desc, cache, x[:, :, :1], x[:, :, 1:], ctx, new_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    assert ctx.tolist() == lens
    q = torch.from_numpy(rng.standard_normal((batch, 2, 64))).to(torch.bfloat16).cuda()
    ws = ops.kv8_attend_workspace(desc, cache)
    ref, ref_lse = ops.kv8_decode_attend(desc, cache, q, ctx, workspace=ws)
    ops.pipeline_check()
    out, lse = ops.kv8_decode_attend(mk(test_wait_timeout=True), cache, q, ctx, workspace=ws)
    with pytest.raises(L.SlsError) as err:
        ops.pipeline_check()
    assert err.value.code == L.SLS_ETIMEOUT
    # that CTA issues no copies any more, so its later rows (of a range; a cluster has one row) have no answer either
    first = next(i for i, n in enumerate(lens) if n)
    keep = ~lse.isnan().any(1).cpu()
    lost = (~keep).nonzero().flatten().tolist()
    assert lost == list(range(first, first + len(lost))) and len(lost) >= 1 and (cap > 4096 or len(lost) == 1)
    assert out[~keep].isnan().all() and lse[~keep].isnan().all()
    assert torch.equal(out[keep], ref[keep]) and torch.equal(lse[keep], ref_lse[keep])
    again, _ = ops.kv8_decode_attend(desc, cache, q, ctx, workspace=ws)
    ops.pipeline_check()
    assert torch.equal(again, ref)
