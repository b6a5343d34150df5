"""Infinite weights of the norm (sls_qk_norm_rope) in channels that are not rotated."""
import numpy as np
import pytest
import torch

from sparse_long_context_gb300 import ops
from tests import kv8_plain as plain
from tests.test_gpu_qk_rope import check, draw, freqs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rot,inter", [(64, 32, False), (64, 32, True), (128, 64, False), (128, 16, True)])
@pytest.mark.parametrize("n,hq,hkv", [(3, 2, 1), (5003, 8, 1), (700, 28, 4)])  # each of the kernel's forms
def test_infinite_weight_shows_in_its_channel_only(dtype, d, rot, inter, n, hq, hkv):
    """y = x w / rms with w infinite: infinite with x's sign, and nothing of it in the neighbouring channels."""
    qkv, (wq, wk) = draw(n + d, n, hq, hkv, d, dtype)
    ch = d - 7
    wq[ch], wk[ch] = float("inf"), float("-inf")
    pos = torch.arange(n, dtype=torch.int32) * 31
    rope = ops.make_rope(hq, hkv, d, dtype, rotary_dim=rot, theta=5e5, interleaved=inter, eps=1e-5)
    dev = qkv.cuda()
    q, k = ops.qk_norm_rope(rope, dev[:, :hq], dev[:, hq:hq + hkv], pos.cuda(), wq.cuda(), wk.cuda())
    x = qkv.double().numpy()
    for got, part, w in ((q, x[:, :hq], wq), (k, x[:, hq:hq + hkv], wk)):
        got = got.cpu()
        w = w.double().numpy().copy()
        assert np.array_equal(got[..., ch].double().numpy(), part[..., ch] * w[ch])
        got[..., ch], w[ch] = 0, 0
        ref, size = plain.norm_rope(part, w, pos.numpy(), rot, inter, freqs(rot, 5e5), 1e-5)
        check(got, ref, size, dtype)
