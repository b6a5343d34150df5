"""Per-head norm and rotation (sls_qk_norm_rope) on the GPU against the plain 64-bit form."""
import numpy as np
import pytest
import torch

from sparse_long_context_gb300 import ops
from tests import kv8_plain as plain

pytestmark = pytest.mark.gpu

# Errors of the kernel's fp32 steps, relative to |y_a| + |y_b| of the channel pair: the mean of D <= 128 squares (at most
# 8 + 5 adds, halved by the root), root, quotient, two products, two products and an add of the rotation, and the sine's
# and cosine's own 2 ulp plus the angle's 2^-24 of half a turn: under 32 steps of 2^-24 = 2^-19.
ARITHMETIC = 2.0 ** -19


def freqs(rot, theta):
    return [theta ** (-2.0 * i / rot) for i in range(rot // 2)]


def check(got, ref, size, dtype):
    got = got.float().cpu().numpy().astype(np.float64)
    tol = ARITHMETIC * size + (torch.finfo(dtype).eps / 2) * np.abs(ref) * (1 + ARITHMETIC) + 1e-37
    assert (np.abs(got - ref) <= tol).all(), np.max(np.abs(got - ref) / tol)


def draw(seed, n, hq, hkv, d, dtype):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn((n, hq + 2 * hkv, d), generator=g) * torch.exp(torch.randn(d, generator=g))).to(dtype)
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(dtype) for _ in range(2)]
    return qkv, w


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (128, 128, True), (64, 64, False), (64, 32, True),
                                         (128, 48, False), (128, 16, False), (64, 16, True), (128, 0, False)])
@pytest.mark.parametrize("n,hq,hkv", [(1, 1, 1), (37, 7, 1), (300, 12, 2)])
def test_matches_plain(dtype, d, rot, inter, n, hq, hkv):
    qkv, (wq, wk) = draw(n + d + rot, n, hq, hkv, d, dtype)
    pos = torch.from_numpy(np.random.default_rng(n).integers(0, 1 << 20, n).astype(np.int32))
    pos[0] = 0 if n > 1 else 2 ** 31 - 1
    rope = ops.make_rope(hq, hkv, d, dtype, rotary_dim=rot, theta=5e5, interleaved=inter, eps=1e-5)
    dev = qkv.cuda()
    q, k = ops.qk_norm_rope(rope, dev[:, :hq], dev[:, hq:hq + hkv], pos.cuda(), wq.cuda(), wk.cuda())
    x = qkv.double().numpy()
    for got, part, w in ((q, x[:, :hq], wq), (k, x[:, hq:hq + hkv], wk)):
        ref, size = plain.norm_rope(part, w.double().numpy(), pos.numpy(), rot, inter, freqs(rot, 5e5), 1e-5)
        check(got, ref, size, dtype)
    assert torch.equal(dev.cpu(), qkv)  # the projection is only read


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (64, 64, True), (64, 16, False), (128, 0, True)])
@pytest.mark.parametrize("hq,hkv", [(8, 1), (7, 1), (5, 0), (0, 3), (4, 4), (13, 2)])
def test_many_tokens_of_few_heads(dtype, d, rot, inter, hq, hkv):
    """Several tokens to a warp, skipped ones among them (the last too), results in place."""
    n = 5003
    qkv, (wq, wk) = draw(d + rot + hq, n, hq, hkv, d, dtype)
    pos = torch.from_numpy(np.random.default_rng(d + hq).integers(0, 2 ** 31, n, dtype=np.int64).astype(np.int32))
    pos[3::11] = -1
    pos[-1] = -5
    rope = ops.make_rope(hq, hkv, d, dtype, rotary_dim=rot, theta=5e5, interleaved=inter, eps=1e-5)
    dev = qkv.cuda()
    q, k = dev[:, :hq] if hq else None, dev[:, hq:hq + hkv] if hkv else None
    ops.qk_norm_rope(rope, q, k, pos.cuda(), wq.cuda() if hq else None, wk.cuda() if hkv else None, q_out=q, k_out=k)
    x = qkv.double().numpy()
    live = pos.numpy() >= 0
    for got, part, w in ((q, x[:, :hq], wq), (k, x[:, hq:hq + hkv], wk)):
        if got is not None:
            ref, size = plain.norm_rope(part[live], w.double().numpy(), pos.numpy()[live], rot, inter, freqs(rot, 5e5), 1e-5)
            check(got.cpu()[live], ref, size, dtype)
    assert torch.equal(dev.cpu()[~live], qkv[~live])
    assert torch.equal(dev[:, hq + hkv:].cpu(), qkv[:, hq + hkv:])


def test_without_norm_given_frequencies_and_one_side():
    qkv, (_, wk) = draw(5, 65, 4, 2, 128, torch.bfloat16)
    pos = torch.arange(65, dtype=torch.int32) * 977
    f = [1.0 / (1 + i) for i in range(32)]
    rope = ops.make_rope(4, 2, 128, torch.bfloat16, rotary_dim=64, inv_freq=f)
    dev = qkv.cuda()
    q, k = ops.qk_norm_rope(rope, dev[:, :4], dev[:, 4:6], pos.cuda(), None, wk.cuda())
    x = qkv.double().numpy()
    check(q, *plain.norm_rope(x[:, :4], None, pos.numpy(), 64, False, f, 0), torch.bfloat16)
    check(k, *plain.norm_rope(x[:, 4:6], wk.double().numpy(), pos.numpy(), 64, False, f, 1e-6), torch.bfloat16)
    only = ops.make_rope(0, 2, 128, torch.bfloat16, rotary_dim=64, inv_freq=f)
    q2, k2 = ops.qk_norm_rope(only, None, dev[:, 4:6], pos.cuda(), None, wk.cuda())
    assert q2 is None and torch.equal(k2, k)


@pytest.mark.parametrize("n", [3, 5003])
@pytest.mark.parametrize("dtype,d,hq,hkv", [(torch.bfloat16, 64, 4, 2), (torch.bfloat16, 64, 3, 5), (torch.bfloat16, 64, 7, 6),
                                            (torch.float32, 64, 3, 1), (torch.float32, 128, 1, 1), (torch.bfloat16, 128, 3, 2)])
@pytest.mark.parametrize("norm_q,norm_k", [(True, False), (False, True), (False, False)])
def test_sides_of_a_step_with_and_without_norm(n, dtype, d, hq, hkv, norm_q, norm_k):
    """Queries and keys next to each other in a warp, one side normalised and the other not; heads first in memory."""
    qkv, (wq, wk) = draw(n + d + hq, n, hq, hkv, d, dtype)
    pos = torch.arange(n, dtype=torch.int32) * 401
    rope = ops.make_rope(hq, hkv, d, dtype, rotary_dim=d // 2, theta=1e4, eps=1e-5)
    dev = qkv.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    q, k = ops.qk_norm_rope(rope, dev[:, :hq], dev[:, hq:hq + hkv], pos.cuda(), wq.cuda() if norm_q else None,
                            wk.cuda() if norm_k else None)
    x = qkv.double().numpy()
    for got, part, w in ((q, x[:, :hq], wq if norm_q else None), (k, x[:, hq:hq + hkv], wk if norm_k else None)):
        ref, size = plain.norm_rope(part, None if w is None else w.double().numpy(), pos.numpy(), d // 2, False,
                                    freqs(d // 2, 1e4), 1e-5)
        check(got, ref, size, dtype)


def test_in_place_strided_skipped_and_empty():
    hq, hkv, d, n = 6, 2, 64, 50
    qkv, (wq, wk) = draw(9, n, hq, hkv, d, torch.bfloat16)
    pos = torch.arange(n, dtype=torch.int32)
    pos[::7] = -1
    rope = ops.make_rope(hq, hkv, d, torch.bfloat16)
    dev = qkv.cuda()
    q, k = ops.qk_norm_rope(rope, dev[:, :hq], dev[:, hq:hq + hkv], pos.clamp(min=0).cuda(), wq.cuda(), wk.cuda())
    ops.qk_norm_rope(rope, dev[:, :hq], dev[:, hq:hq + hkv], pos.cuda(), wq.cuda(), wk.cuda(),
                     q_out=dev[:, :hq], k_out=dev[:, hq:hq + hkv])
    live = pos >= 0
    assert torch.equal(dev[:, :hq].cpu()[live], q.cpu()[live])
    assert torch.equal(dev[:, hq:hq + hkv].cpu()[live], k.cpu()[live])
    assert torch.equal(dev.cpu()[~live], qkv[~live])           # skipped tokens keep their contents
    assert torch.equal(dev[:, hq + hkv:].cpu(), qkv[:, hq + hkv:])
    # heads-first outputs
    out = torch.zeros((hq, n, d), dtype=torch.bfloat16, device="cuda")
    ops.qk_norm_rope(rope, qkv.cuda()[:, :hq], qkv.cuda()[:, hq:hq + hkv], pos.clamp(min=0).cuda(), wq.cuda(), wk.cuda(),
                     q_out=out.transpose(0, 1))
    assert torch.equal(out.transpose(0, 1), q)
    # a single token's or head's stride does not matter, whatever the view says
    odd = torch.as_strided(qkv.cuda()[0], (1, hq, d), (13, d, 1))
    one, _ = ops.qk_norm_rope(rope, odd, qkv.cuda()[:1, hq:hq + hkv], pos[:1].clamp(min=0).cuda(), wq.cuda(), wk.cuda())
    assert torch.equal(one[0], q[0])
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    q0, k0 = ops.qk_norm_rope(rope, dev[:0, :hq], dev[:0, hq:hq + hkv], none)
    assert q0.shape == (0, hq, d) and k0.shape == (0, hkv, d)


def test_zero_rows_infinities_and_nan_stay_in_their_head():
    qkv, (wq, wk) = draw(3, 40, 4, 1, 128, torch.bfloat16)
    qkv[3, 0] = 0
    qkv[4, 1, 5] = float("inf")
    qkv[5, 2, 9] = float("nan")
    rope = ops.make_rope(4, 1, 128, torch.bfloat16)
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    dev = qkv.cuda()
    q, _ = ops.qk_norm_rope(rope, dev[:, :4], dev[:, 4:5], pos, wq.cuda(), wk.cuda())
    assert (q[3, 0] == 0).all()
    assert q[5, 2].isnan().all()
    bad = torch.zeros((40, 4), dtype=torch.bool)
    bad[4, 1] = bad[5, 2] = True
    assert q.cpu()[~bad].isfinite().all()


@pytest.mark.parametrize("inter", [False, True])
def test_channels_that_are_not_rotated_pass_an_infinity_alone(inter):
    x = torch.ones((2, 1, 64), dtype=torch.bfloat16)
    x[0, 0, 37] = float("inf")
    x[1, 0, 33] = float("nan")
    rope = ops.make_rope(1, 0, 64, torch.bfloat16, rotary_dim=32, interleaved=inter)
    y = ops.qk_norm_rope(rope, x.cuda(), None, torch.tensor([3, 0], dtype=torch.int32, device="cuda"))[0].cpu()
    assert torch.equal(y[0, 0, 32:], x[0, 0, 32:]) and y[0, 0, :32].isfinite().all()
    assert y[1, 0, 33].isnan() and y[1].isnan().sum() == 1


def test_other_stream_and_graph():
    qkv, (wq, wk) = draw(11, 33, 4, 2, 128, torch.bfloat16)
    rope = ops.make_rope(4, 2, 128, torch.bfloat16)
    pos = torch.arange(33, dtype=torch.int32, device="cuda")
    dev, w = qkv.cuda(), wq.cuda()
    ref, _ = ops.qk_norm_rope(rope, dev[:, :4], dev[:, 4:6], pos, w, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, _ = ops.qk_norm_rope(rope, dev[:, :4], dev[:, 4:6], pos, w, w)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, ref)
    qo, ko = torch.zeros_like(ref), torch.zeros((33, 2, 128), dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.qk_norm_rope(rope, dev[:, :4], dev[:, 4:6], pos, w, w, q_out=qo, k_out=ko)
    g.replay()
    assert torch.equal(qo, ref)
    pos += 5
    g.replay()
    assert torch.equal(qo, ops.qk_norm_rope(rope, dev[:, :4], dev[:, 4:6], pos, w, w)[0])
