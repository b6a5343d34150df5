"""The decode step over a paged cache (ops.PagedDecode) and its replayed loop: prompts, steps, forks, cuts, frees and
compactions together, against the plain form of every step; pools and rows at the limits."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from sparse_long_context_gb300 import _lib as L
from sparse_long_context_gb300 import harness, ops
from tests import paged_plain as plain
from tests.test_gpu_paged import BF16, F32, Pair, ints, same

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Run:
    """A step and its plain form.  The rotated queries and keys are the kernel's (qk_norm_rope has tests of its own)."""

    def __init__(self, batch, hq, hkv, d, page, cap, pool, dtype=BF16, seed=0, **kw):
        self.desc = ops.make_desc(batch, hq, hkv, d, page, cap, dtype)
        self.rng = np.random.default_rng(seed)
        self.dtype = dtype
        rope = ops.make_rope(hq, hkv, d, dtype, theta=1e4)
        weights = [torch.from_numpy(1 + 0.2 * self.rng.standard_normal(d)).to(dtype).cuda() for _ in range(2)]
        self.step = ops.PagedDecode(self.desc, rope, pool, q_weight=weights[0], k_weight=weights[1], **kw)
        c = self.step.cache
        self.plain = plain.PlainPaged(batch, hkv, d, page, cap, c.k_pages, c.v_pages, c.kmin, c.kmax)

    def qkv(self, *shape):
        d = self.desc
        x = self.rng.standard_normal((*shape, d.num_q_heads + 2 * d.num_kv_heads, d.head_dim))
        return torch.from_numpy(x).to(self.dtype).cuda()

    def prefill(self, lens):
        d, s = self.desc, self.step
        x = self.qkv(d.batch, max([*lens, 1]))
        at = s.ctx_len.clone()
        q = s.prefill(x, ints(lens))
        pos = at[:, None] + torch.arange(x.shape[1], dtype=torch.int32, device="cuda")
        k = x[:, :, d.num_q_heads:d.num_q_heads + d.num_kv_heads].reshape(-1, d.num_kv_heads, d.head_dim)
        k = ops.qk_norm_rope(ops.make_rope(0, d.num_kv_heads, d.head_dim, self.dtype, theta=1e4), None, k.contiguous(),
                             pos.reshape(-1), k_weight=s.k_weight)[1].view(d.batch, -1, d.num_kv_heads, d.head_dim)
        want = self.plain.append(k, x[:, :, d.num_q_heads + d.num_kv_heads:], lens)
        assert s.pos.tolist() == want
        self.check()
        return q

    def decoded(self, x, out, lse, sink):
        """What a step did with the projected heads x, in plain form."""
        d, s = self.desc, self.step
        want = self.plain.append(s.k_new[:, None], x[:, None, d.num_q_heads + d.num_kv_heads:], [1] * d.batch)
        assert s.pos.tolist() == want
        self.check()
        lists = None if s.page_idx is None else s.page_idx.tolist()
        want = self.plain.attend(s.q, 1 / math.sqrt(d.head_dim), lists, sink)
        tol, tol_lse = plain.bounds(self.dtype, d.head_dim, want[0], *want[2:])
        assert bool(((out.cpu().double() - want[0]).abs() <= tol).all())
        live = want[1].isfinite()
        assert bool(((lse.cpu().double() - want[1])[live].abs() <= (tol_lse + want[1].abs() * 2.0 ** -22)[live]).all())
        if lists is not None:  # the selection of the rows' own summaries
            at = s.cache.table.clamp(min=0).long()
            lo, hi = (y[at].transpose(1, 2).contiguous() for y in (s.cache.kmin, s.cache.kmax))
            assert torch.equal(ops.select_pages(d, s.q, lo, hi, s.ctx_len, s.k, s.n_sink, s.n_local), s.page_idx)

    def decode(self, sink=None):
        x = self.qkv(self.desc.batch)
        self.decoded(x, *self.step(x, sink), sink)

    def fork(self, parent, keep=None):
        done = self.step.fork(ints(parent), None if keep is None else ints(keep)).item()
        assert done == int(self.plain.fork(parent, keep))
        self.check()

    def compact(self):
        self.step.compact()
        self.plain.compact()
        self.check()

    def check(self):
        p, c = self.plain, self.step.cache
        assert c.ctx_len.tolist() == p.ctx and torch.equal(c.table.cpu(), p.table()) and c.refs.tolist() == p.refs()
        assert same(c.k_pages, p.k) and same(c.v_pages, p.v)
        if p.lo is not None:
            assert same(c.kmin, p.lo) and same(c.kmax, p.hi)
        ops.pipeline_check()


@pytest.mark.parametrize("dtype,d,page,kw", [(BF16, 128, 16, {}), (BF16, 64, 16, dict(k_budget=6, n_sink_pages=1, n_local_tokens=20)),
                                             (F32, 64, 32, {}), (F32, 128, 16, dict(k_budget=5, n_sink_pages=1, n_local_tokens=16))])
def test_prompts_steps_forks_and_compactions_together(dtype, d, page, kw):
    run = Run(5, 6, 2, d, page, 24 * page, 70, dtype, **kw)
    sink = torch.randn(6, device="cuda")
    run.prefill([9 * page + 3, 5, 0, 4 * page, 0])
    for _ in range(3):
        run.decode()
    run.prefill([0, 3 * page, 7, 0, 0])
    run.fork([0, 1, 0, 3, 3], [999, 999, 4 * page, 999, 2 * page + 1])  # two forks of prompts, at and inside pages
    for _ in range(page + 2):
        run.decode(sink)
    run.fork([2, 2, 0, -1, 4])            # beams
    run.compact()
    run.decode()
    run.fork([0, 1, 2, 3, 4], [page, 2 * page + 5, 999, 999, 1])  # drafts taken back
    run.decode(sink)
    run.fork([-1] * 5)
    run.decode()
    run.prefill([page] * 5)


def test_replayed_loop_with_forks_between_the_replays():
    run = Run(4, 8, 2, 128, 16, 512, 60, k_budget=8, n_sink_pages=1, n_local_tokens=32)
    run.prefill([200, 17, 100, 0])
    loop = harness.PagedDecodeLoop(run.step)
    loop.capture()
    run.check()
    for step in range(40):
        x = run.qkv(4)
        loop.qkv.copy_(x)
        out, lse = loop.replay()
        run.decoded(x, out, lse, None)
        if step == 10:
            run.fork([0, 0, 2, 2], [999, 150, 999, 50])
        if step == 20:
            run.fork([1, 0, 3, 2])
            run.compact()
        if step == 30:
            run.fork([0, -1, 2, 3])


def test_a_step_for_whose_tokens_the_pool_lacks_pages():
    run = Run(3, 4, 1, 64, 16, 256, 4)
    run.prefill([16, 15, 31])   # all four pages
    run.decode()                # sequence 0 needs one more: left as it is; the others go on
    assert run.step.pos.tolist() == [-1, 15, 31]
    run.fork([0, -1, 2])
    run.decode()
    assert run.step.pos.tolist() == [16, -1, -1] or run.step.ctx_len.tolist()[0] == 17


def test_a_step_with_a_bad_argument_appends_nothing():
    run = Run(2, 4, 2, 64, 16, 256, 20)
    x, sink = run.qkv(2), torch.zeros(4, device="cuda")
    for args in ((x, sink[:-1]), (x, sink.double()), (x, sink.cpu()), (x[:1], None), (x[:, :-1], None)):
        with pytest.raises(ValueError):
            run.step(*args)
        run.check()


def test_arguments_of_another_shape_type_or_device_are_refused():
    pair = Pair(2, 4, 2, 64, 16, 256, 20)
    d, c = pair.desc, pair.cache
    kv, q = pair.new((2, 3, 2, 64)).cuda(), pair.new((2, 4, 64)).cuda()
    bad = [lambda: ops.paged_append(d, c, kv.float(), kv.float()), lambda: ops.paged_append(d, c, kv[:1], kv[:1]),
           lambda: ops.paged_append(d, c, kv, kv[:, :2]), lambda: ops.paged_append(d, c, kv.cpu(), kv.cpu()),
           lambda: ops.paged_append(d, c, kv, kv, new_len=ints([1])), lambda: ops.paged_append(d, c, kv, kv, new_len=ints([1, 1]).long()),
           lambda: ops.paged_append(d, c, kv.transpose(2, 3), kv), lambda: ops.paged_decode_attend(d, c, q.float()),
           lambda: ops.paged_decode_attend(d, c, q[:, :3]), lambda: ops.paged_decode_attend(d, c, q, page_idx=ints([[1]])),
           lambda: ops.paged_decode_attend(d, c, q, sink=q[0, :, 0]), lambda: ops.paged_fork(d, c, ints([0])),
           lambda: ops.paged_fork(d, c, ints([0, 1]), keep_len=ints([0])), lambda: ops.paged_fork(d, c, torch.tensor([0, 1])),
           lambda: ops.paged_compact(d, c, moved=ints([0])), lambda: ops.paged_select_pages(d, c, q.float(), 3),
           lambda: ops.paged_select_pages(d, c, q, 3, out=ints([[0, 0, 0]])),
           lambda: ops.paged_append(ops.make_desc(2, 4, 2, 64, 16, 512, BF16), c, kv, kv),
           lambda: ops.PagedCache(d, c.k_pages, c.v_pages[:3]), lambda: ops.PagedCache(d, c.k_pages, c.v_pages, kmin=c.kmin),
           lambda: ops.PagedCache(d, c.k_pages.float(), c.v_pages.float())]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(L.SlsError):
        ops.paged_append(d, c, kv[:, :, :, ::1].as_strided((2, 3, 2, 64), (384, 128, 60, 1)), kv)
    pair.check()


def test_pools_beyond_four_gigabytes():
    """Pages whose bytes lie past 2^32, and rows past 2^24: appended, selected, attended, forked and compacted."""
    pool, hkv, d = 140000, 8, 128  # 4.6 GB each of keys and values
    desc = ops.make_desc(3, 16, hkv, d, 16, 1 << 21, BF16)
    zeros = torch.zeros((pool, hkv, 16, d), dtype=BF16, device="cuda")
    meta = torch.zeros((pool, hkv, d), dtype=BF16, device="cuda")
    cache = ops.PagedCache(desc, zeros, torch.zeros_like(zeros), meta, torch.zeros_like(meta))
    # all but the last 60 pages belong to sequence 0
    table = torch.full((3, 1 << 17), -1, dtype=torch.int32, device="cuda")
    table[0, :131072] = torch.arange(131072, dtype=torch.int32, device="cuda")
    cache.load(table, ints([1 << 21, 0, 0]))
    held = torch.arange(131072, pool - 60, dtype=torch.int32, device="cuda")
    table[1, :held.numel()] = held
    cache.load(table, ints([1 << 21, 16 * held.numel(), 0]))
    ops.pipeline_check()
    g = torch.Generator("cuda").manual_seed(1)
    kv = torch.randn((3, 700, hkv, d), generator=g, device="cuda").to(BF16)
    ops.paged_append(desc, cache, kv, kv.flip(1), new_len=ints([0, 0, 700]))
    assert cache.table[2, :44].tolist() == list(range(pool - 60, pool - 16))
    k, v = cache.values(2)
    assert same(k, kv[2].transpose(0, 1)) and same(v, kv[2].flip(0).transpose(0, 1))
    ops.paged_fork(desc, cache, ints([-1, 2, 2]), ints([0, 333, 700]))
    assert cache.table[1, 20].item() == pool - 16
    q = torch.randn((3, 16, d), generator=g, device="cuda").to(BF16)
    idx = ops.paged_select_pages(desc, cache, q, 50)
    before = ops.paged_decode_attend(desc, cache, q)
    listed = ops.paged_decode_attend(desc, cache, q, page_idx=idx)
    ops.paged_compact(desc, cache)
    assert cache.table[2, :44].tolist() == list(range(44)) and cache.table[1, 20].item() == 44  # in order: the copy came last
    after = ops.paged_decode_attend(desc, cache, q)
    assert same(before[0], after[0]) and same(before[1], after[1]) and same(listed[0], ops.paged_decode_attend(desc, cache, q, page_idx=idx)[0])
    ops.pipeline_check()
    p = plain.PlainPaged(3, hkv, d, 16, 1 << 21, cache.k_pages[:45], cache.v_pages[:45])
    p.rows, p.ctx = [[], cache.table[1, :21].tolist(), cache.table[2, :44].tolist()], [0, 333, 700]
    want = p.attend(q, 1 / math.sqrt(d))
    tol, _ = plain.bounds(BF16, d, want[0], *want[2:])
    assert bool(((after[0].cpu().double() - want[0]).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_over_4096_rows(dtype):
    pair = Pair(1024, 8, 4, 64, 16, 128, 2600, dtype, summaries=False)
    pair.append([int(n) for n in pair.rng.integers(0, 60, 1024)])
    pair.attend()


def test_one_workspace_for_calls_of_several_shapes():
    a, b = (Pair(n, 8, 2, 128, 16, cap, 700, summaries=False, seed=n) for n, cap in ((3, 4096), (12, 1024)))
    a.append([3000, 1, 2999])
    b.append([int(n) for n in b.rng.integers(0, 900, 12)])
    ws = max(ops.paged_attend_workspace(a.desc, a.cache), ops.paged_attend_workspace(b.desc, b.cache), key=lambda t: t.numel())
    for _ in range(3):
        a.attend(workspace=ws)
        b.attend(workspace=ws)


def test_first_calls_of_a_process_captured_in_a_graph():
    code = """
import torch
from sparse_long_context_gb300 import ops
desc = ops.make_desc(2, 4, 2, 64, 16, 256, torch.bfloat16)
step = ops.PagedDecode(desc, ops.make_rope(4, 2, 64, torch.bfloat16), 40, k_budget=4)
x = torch.randn(2, 8, 64, device="cuda").to(torch.bfloat16)
parent = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step(x)
    step.fork(parent)
    step.compact()
for n in range(1, 40):
    graph.replay()
    assert step.ctx_len.tolist() == [n, n], step.ctx_len
assert torch.equal(step.out[0], step.out[0]) and step.out.isfinite().all() and step.done.item() == 1
ops.pipeline_check()
print("fine")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cap", [512, 8192])
def test_values_that_are_not_finite_stay_in_their_channel_or_head(dtype, cap):
    """(In a cluster and in ranges.)  A key of -inf or of the type's lowest value takes its token out; NaN and infinite values show
    in their channel, a NaN query in its head."""
    pair = Pair(3, 8, 2, 64, 16, cap, 3 * cap // 16, dtype, summaries=False)
    pair.append([cap - 3, 200, 33])
    q = pair.new((3, 8, 64))
    q[:, :, 5] = q[:, :, 5].abs() + 0.5   # channel 5 of every query is positive
    page = lambda b, t: (pair.plain.rows[b][t // 16], t % 16)  # noqa: E731
    for b, t, x in ((0, 7, -math.inf), (0, 100, torch.finfo(dtype).min), (1, 199, -math.inf), (2, 0, torch.finfo(dtype).min)):
        p, r = page(b, t)
        for side in (pair.plain.k, pair.cache.k_pages):
            side[p, :, r, 5] = x
    want, lse, size, dots, count = pair.plain.attend(q, 0.125)
    pair.plain.k[pair.plain.k.isinf()] = 0     # for the tolerances: the tokens' own scores are exact
    pair.plain.k[pair.plain.k == torch.finfo(dtype).min] = 0
    dots = pair.plain.attend(q, 0.125)[3]
    tol, tol_lse = plain.bounds(dtype, 64, want, size, dots, count)
    out, got = ops.paged_decode_attend(pair.desc, pair.cache, q.cuda())
    assert bool(((out.cpu().double() - want).abs() <= tol).all()) and bool(((got.cpu().double() - lse).abs() <= tol_lse + 1e-5).all())
    # NaN and infinities among the values of the newest token but one (whose weights are above zero), a NaN query
    for b, x, ch in ((0, math.nan, 3), (1, math.inf, 40), (2, -math.inf, 63)):
        p, r = page(b, pair.plain.ctx[b] - 2)
        pair.cache.v_pages[p, 1, r, ch] = x
    q[2, 1, 0] = math.nan
    odd, odd_lse = ops.paged_decode_attend(pair.desc, pair.cache, q.cuda())
    hit = torch.zeros_like(odd, dtype=torch.bool)
    hit[0, 4:, 3] = hit[1, 4:, 40] = hit[2, 4:, 63] = hit[2, 1] = True
    assert torch.equal(odd.isfinite(), ~hit) and torch.equal(odd[~hit], out[~hit])
    assert odd[0, 4:, 3].isnan().all() and bool((odd[1, 4:, 40] == math.inf).all()) and bool((odd[2, 4:, 63] == -math.inf).all())
    assert odd_lse[2, 1].isnan() and odd_lse.isnan().sum() == 1


def test_sinks_of_every_size():
    pair = Pair(2, 4, 2, 64, 16, 256, 40, summaries=False)
    pair.append([100, 0])
    q = pair.new((2, 4, 64))
    none = ops.paged_decode_attend(pair.desc, pair.cache, q.cuda())
    out, lse = ops.paged_decode_attend(pair.desc, pair.cache, q.cuda(), sink=torch.full((4,), -math.inf, device="cuda"))
    assert same(out, none[0]) and same(lse, none[1])
    pair.attend(q, sink=torch.tensor([-1e30, 0.0, 20.0, 1e4]))


def test_two_caches_on_two_streams():
    pairs = [Pair(4, 8, 2, 128, 16, 2048, 400, seed=s) for s in range(2)]
    streams = [torch.cuda.Stream() for _ in pairs]
    outs = []
    for _ in range(4):
        for pair in pairs:
            pair.kv = pair.new((4, 60, 4, 128))
            pair.dev, pair.q = pair.kv.cuda(), pair.new((4, 8, 128)).cuda()
        torch.cuda.synchronize()
        outs = []
        for pair, stream in zip(pairs, streams):
            with torch.cuda.stream(stream):
                ops.paged_append(pair.desc, pair.cache, pair.dev[:, :, :2], pair.dev[:, :, 2:])
                ops.paged_fork(pair.desc, pair.cache, torch.tensor([1, 0, 2, 2], dtype=torch.int32, device="cuda"))
                idx = ops.paged_select_pages(pair.desc, pair.cache, pair.q, 3, 1)
                outs.append((ops.paged_decode_attend(pair.desc, pair.cache, pair.q, page_idx=idx), idx))
                ops.paged_compact(pair.desc, pair.cache)
        torch.cuda.synchronize()
        for pair, ((out, _), idx) in zip(pairs, outs):
            pair.plain.append(pair.kv[:, :, :2], pair.kv[:, :, 2:], [60] * 4)
            assert pair.plain.fork([1, 0, 2, 2], None)
            pair.plain.compact()
            pair.check()
            want = pair.plain.attend(pair.q, 1 / math.sqrt(128), idx.tolist())
            tol, _ = plain.bounds(BF16, 128, want[0], *want[2:])
            assert bool(((out.cpu().double() - want[0]).abs() <= tol).all())
