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
