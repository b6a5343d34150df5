"""The 8-bit attend's bounded waits (the planted never-completing phase of SLS_FLAG_TEST_WAIT_TIMEOUT; no copy is
issued for it)."""
import numpy as np
import pytest
import torch

from sparse_long_context_gb300 import _lib as L
from sparse_long_context_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cap", [4096, 1 << 20])  # a cluster per row; ranges over all rows
def test_wait_timeout_poisons_the_first_row_only(cap):
    rng = np.random.default_rng(0)
    mk = lambda **kw: ops.make_desc(4, 6, 1, 128, 16, cap, torch.bfloat16, **kw)  # noqa: E731
    desc = mk()
    cache = ops.Kv8Cache.empty(desc, "int8", 64)
    ctx = torch.zeros(4, dtype=torch.int32, device="cuda")
    x = torch.from_numpy(rng.standard_normal((4, 4000, 2, 128))).to(torch.bfloat16).cuda()
    ops.kv8_append(desc, cache, x[:, :, :1], x[:, :, 1:], ctx)
    q = torch.from_numpy(rng.standard_normal((4, 6, 128))).to(torch.bfloat16).cuda()
    ws = ops.kv8_attend_workspace(desc, cache)
    ref, ref_lse = ops.kv8_decode_attend(desc, cache, q, ctx, workspace=ws)
    ops.pipeline_check()
    out, lse = ops.kv8_decode_attend(mk(test_wait_timeout=True), cache, q, ctx, workspace=ws)
    with pytest.raises(L.SlsError) as err:
        ops.pipeline_check()
    assert err.value.code == L.SLS_ETIMEOUT
    assert out[0].isnan().all() and lse[0].isnan().all()
    assert torch.equal(out[1:], ref[1:]) and torch.equal(lse[1:], ref_lse[1:])
    again, _ = ops.kv8_decode_attend(desc, cache, q, ctx, workspace=ws)
    ops.pipeline_check()
    assert torch.equal(again, ref)
