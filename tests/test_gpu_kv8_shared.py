"""One workspace of the 8-bit attend for calls of different shapes, one after the other."""
import numpy as np
import pytest
import torch

from sparse_long_context_gb300 import ops
from tests.test_gpu_kv8 import bf16

pytestmark = pytest.mark.gpu


def setup(batch, cap, d, lens, seed):
    rng = np.random.default_rng(seed)
    desc = ops.make_desc(batch, 4, 1, d, 16, cap, torch.bfloat16)
    cache = ops.Kv8Cache.empty(desc, "int8", 64)
    ctx = torch.zeros(batch, dtype=torch.int32, device="cuda")
    x = torch.randn((batch, max(lens), 2, d), generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(torch.bfloat16)
    ops.kv8_append(desc, cache, x[:, :, :1], x[:, :, 1:], ctx, new_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    return desc, cache, bf16(rng, (batch, 4, d)).cuda(), ctx


@pytest.mark.parametrize("mass", [False, True])
def test_workspace_shared_by_calls_of_different_shapes(mass):
    """Both shapes go in ranges over all rows (deep capacities): partials of the one call may not lie where the other one's
    arrival counters are."""
    few = setup(32, 65536, 64, [5000 + 31 * i for i in range(32)], 1)
    many = setup(256, 16384, 64, [(137 * i) % 2000 for i in range(256)], 2)
    ws = ops.kv8_attend_workspace(many[0], many[1], mass)
    own = ops.kv8_attend_workspace(few[0], few[1], mass)
    if own.numel() > ws.numel():
        ws = torch.zeros_like(own)

    def call(s, workspace):
        desc, cache, q, ctx = s
        out = torch.full_like(q, -77.0)
        sums = torch.zeros((desc.batch, 1, desc.capacity // 64), device="cuda") if mass else None
        got = ops.kv8_decode_attend(desc, cache, q, ctx, out=out, mass_out=sums, workspace=workspace)
        return [*got] + ([sums] if mass else [])

    want = {i: call(s, None) for i, s in enumerate((few, many))}  # each on a workspace of its own
    ops.pipeline_check()
    for i in (0, 1, 0, 1, 1, 0):
        for got, ref in zip(call((few, many)[i], ws), want[i]):
            assert torch.equal(got, ref), i
    ops.pipeline_check()
