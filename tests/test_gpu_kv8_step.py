"""The decode step over the 8-bit cache (ops.Kv8Decode): pieces of prompts of every shape."""
import numpy as np
import pytest
import torch

from sparse_long_context_gb300 import ops
from tests.test_gpu_kv8 import bf16, ints, same

pytestmark = pytest.mark.gpu

B, HQ, H, D = 2, 6, 2, 64


def step(**kw):
    desc = ops.make_desc(B, HQ, H, D, 16, 256, torch.bfloat16)
    return ops.Kv8Decode(desc, ops.make_rope(HQ, H, D, torch.bfloat16), "int8", 16, **kw)


def held(s):
    return [s.ctx_len, s.cache.k_codes, s.cache.v_codes, s.cache.k_scales, s.cache.v_scales, s.cache.k_tail, s.cache.v_tail]


def test_prefill_of_an_empty_piece():
    s = step(mass=True)
    qkv = bf16(np.random.default_rng(0), (B, 40, HQ + 2 * H, D)).cuda()
    assert s.prefill(qkv[:, :0].contiguous()).shape == (B, 0, HQ, D)
    s.prefill(qkv)
    before = [x.clone() for x in held(s)]
    assert s.prefill(qkv[:, :0].contiguous(), ints([0, 3])).shape == (B, 0, HQ, D)
    assert s.ctx_len.tolist() == [40, 40] and all(same(x, y) for x, y in zip(held(s), before))


def test_prefill_in_slices_of_one_batch_equals_the_whole():
    """The pieces are strided views [B, T, heads, D] of one projection's output, ragged lengths among them."""
    a, b = step(), step()
    qkv = bf16(np.random.default_rng(1), (B, 90, HQ + 2 * H, D)).cuda()
    whole = a.prefill(qkv)
    parts = [b.prefill(qkv[:, lo:hi]) for lo, hi in ((0, 33), (33, 34), (34, 90))]
    assert torch.equal(torch.cat(parts, 1), whole)
    for x, y in zip(held(a)[:-2], held(b)[:-2]):
        assert same(x, y)
    assert same(a.cache.k_tail[:, :, :10], b.cache.k_tail[:, :, :10])
    wide = torch.zeros((B, 7, HQ + 2 * H + 3, D), dtype=torch.bfloat16, device="cuda")
    wide[:, :, 1:-2] = bf16(np.random.default_rng(2), (B, 7, HQ + 2 * H, D)).cuda()
    x = a.prefill(wide[:, :, 1:-2], ints([7, 2]))  # heads that are a slice, too
    y = b.prefill(wide[:, :, 1:-2].contiguous(), ints([7, 2]))
    assert torch.equal(x[0], y[0]) and torch.equal(x[1, :2], y[1, :2]) and a.ctx_len.tolist() == [97, 92]
    assert same(a.cache.k_tail[:, :, :1], b.cache.k_tail[:, :, :1]) and same(a.cache.k_codes, b.cache.k_codes)


@pytest.mark.parametrize("kw", [dict(dtype=torch.float32), dict(batch=4097)])
def test_step_of_a_shape_that_the_attend_does_not_take_is_refused(kw):
    dt = kw.get("dtype", torch.bfloat16)
    desc = ops.make_desc(kw.get("batch", 1), 2, 1, 64, 16, 16, dt)
    with pytest.raises(ValueError, match="does not take"):
        ops.Kv8Decode(desc, ops.make_rope(2, 1, 64, dt), "int8", 16)


def test_refused_eviction_leaves_the_positions():
    s = step(mass=True)
    s.prefill(bf16(np.random.default_rng(4), (B, 100, HQ + 2 * H, D)).cuda(), ints([100, 20]))
    for bad in ((0, 0, 0), (4, 3, 2), (16, 0, 0)):
        with pytest.raises(ops.L.SlsError):
            s.evict(*bad)
        assert s.evicted.tolist() == [0, 0] and s.ctx_len.tolist() == [100, 20]
    s.evict(3)
    assert s.evicted.tolist() == [48, 0] and s.ctx_len.tolist() == [52, 20]


def test_step_with_a_bad_argument_appends_nothing():
    s = step()
    qkv = bf16(np.random.default_rng(5), (B, HQ + 2 * H, D)).cuda()
    sink = torch.zeros(HQ, device="cuda")
    for args in ((qkv, sink[:-1]), (qkv, sink.double()), (qkv, sink.cpu()), (qkv[:1], None), (qkv[:, :-1], None)):
        with pytest.raises(ValueError):
            s(*args)
        assert s.ctx_len.tolist() == [0, 0]
    s(qkv, sink)
    assert s.ctx_len.tolist() == [1, 1]
