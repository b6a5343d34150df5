"""A sink on another device than the step's is refused before the step changes anything (on stand-ins: no GPU is used)."""
from types import SimpleNamespace

import pytest
import torch

from sparse_long_context_gb300 import _lib as L
from sparse_long_context_gb300 import ops


class Elsewhere:
    """What a step looks at of a tensor on device 1."""
    is_cuda, dtype, shape, device = True, torch.float32, (4,), torch.device("cuda", 1)

    def is_contiguous(self):
        return True

    def get_device(self):
        return 1


@pytest.mark.parametrize("kind", [ops.PagedDecode, ops.Kv8Decode])
def test_a_sink_on_another_device(monkeypatch, kind):
    changed = []
    for name in ("qk_norm_rope", "paged_append", "kv8_append", "paged_select_pages", "select_pages", "paged_decode_attend",
                 "kv8_decode_attend"):
        monkeypatch.setattr(ops, name, lambda *a, _n=name, **k: changed.append(_n))
    step = kind.__new__(kind)
    step.desc = L.AttnDesc(2, 4, 2, 64, 16, 256, L.SLS_DTYPE_BF16, 0, 0.0)
    step.cache = SimpleNamespace(index=0, ctx_len=None)
    step.k = 0
    for name in ("rope", "q_weight", "k_weight", "q", "out", "lse", "pos", "kmin", "kmax", "mass", "page_idx", "workspace"):
        setattr(step, name, None)
    step.k_new = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    if kind is ops.Kv8Decode:
        step.ctx_len = step.evicted = step.positions = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        step(torch.zeros((2, 8, 64), dtype=torch.bfloat16), sink=Elsewhere())
    assert not changed
