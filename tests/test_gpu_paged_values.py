"""The paged cache where its other tests compare calls with each other: lists cut by count and k_fixed, steps captured in a graph and
the positions of a step, against the plain form; tables and lengths of 64 bits; repeated calls."""
import math

import numpy as np
import pytest
import torch

from sparse_long_context_gb300 import _lib as L
from sparse_long_context_gb300 import ops
from tests import paged_plain as plain
from tests.test_gpu_paged import BF16, F32, SHAPES, Pair, ints, same
from tests.test_gpu_paged_step import Run

pytestmark = pytest.mark.gpu


def check(pair, q, lists, got, sink=None):
    """An attend's outputs against the plain form over `lists`."""
    d = pair.desc
    want = pair.plain.attend(q, 1 / math.sqrt(d.head_dim), lists, sink)
    tol, tol_lse = plain.bounds(pair.dtype, d.head_dim, want[0], *want[2:])
    out, lse = (x.cpu().double() for x in got)
    assert bool(((out - want[0]).abs() <= tol).all()), float(((out - want[0]).abs() / tol).max())
    dead = want[1].isinf()
    assert torch.equal(lse[dead], want[1][dead])
    assert bool(((lse - want[1])[~dead].abs() <= (tol_lse + want[1].abs() * 2.0 ** -22)[~dead]).all())


@pytest.mark.parametrize("batch,hkv,d,page,dtype", SHAPES)
def test_lists_cut_by_count_and_k_fixed(batch, hkv, d, page, dtype):
    g, width, rows = 1 + batch % 5, 16, batch * hkv
    pair = Pair(batch, hkv * g, hkv, d, page, 16 * page, batch * 16, dtype, summaries=False, seed=3)
    pair.append([int(n) for n in pair.rng.integers(1, 16 * page, batch)])
    lists = [pair.rng.permutation(16).tolist() for _ in range(rows)]
    for r in range(0, rows, 3):
        lists[r][2] = -1
    q, sink = pair.new((batch, hkv * g, d), 2.0), torch.randn(hkv * g)
    count = [int(n) for n in pair.rng.integers(-1, width + 3, rows)]
    cut = [x[:max(n, 0)] for x, n in zip(lists, count)]
    run = lambda **kw: ops.paged_decode_attend(pair.desc, pair.cache, q.cuda(), page_idx=ints(lists), **kw)  # noqa: E731
    check(pair, q, cut, run(count=ints(count)))
    check(pair, q, cut, run(count=ints(count), sink=sink.cuda()), sink)
    check(pair, q, cut, run(count=ints(count), k_fixed=1))  # count wins
    for k in (1, 2, 7, 15, 16):
        check(pair, q, [x[:k] for x in lists], run(k_fixed=k))
    check(pair, q, [[]] * rows, run(k_fixed=0))
    for k in (-1, width + 1):
        with pytest.raises(L.SlsError):
            run(k_fixed=k)
    ops.pipeline_check()


def test_positions_of_a_step_for_whose_tokens_the_pool_lacks_pages():
    run = Run(3, 4, 1, 64, 16, 256, 4)
    run.prefill([16, 15, 31])
    run.decode()                # sequence 0 needs a page and there is none; the others' tokens have room
    assert run.step.pos.tolist() == [-1, 15, 31] and run.step.ctx_len.tolist() == [16, 16, 32]
    run.fork([0, -1, 2])        # one page free, which sequence 0 takes; sequence 1 has none and needs one, 2 as well
    run.decode()
    assert run.step.pos.tolist() == [16, -1, -1] and run.step.ctx_len.tolist() == [17, 0, 32]


def test_a_captured_run_gives_what_the_same_run_gives_without_a_graph():
    """Steps, forks and compactions replayed from one graph and made one by one: equal outputs, positions, pages and lists."""
    rng = np.random.default_rng(2)
    parent = ints([0, 0, 1])

    def step():
        d = ops.make_desc(3, 4, 2, 64, 16, 256, BF16)
        return ops.PagedDecode(d, ops.make_rope(4, 2, 64, BF16), 60, k_budget=4, n_sink_pages=1, n_local_tokens=16)

    one, two = step(), step()
    buf = torch.zeros((3, 8, 64), dtype=BF16, device="cuda")

    def pass_of(s):
        s(buf)
        s.fork(parent)
        s.compact()

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pass_of(one)
    p = plain.PlainPaged(3, 2, 64, 16, 256, two.cache.k_pages, two.cache.v_pages, two.cache.kmin, two.cache.kmax)
    for _ in range(40):
        buf.copy_(torch.from_numpy(rng.standard_normal((3, 8, 64))).to(BF16))
        graph.replay()
        two(buf)
        # the eager side against the plain form, before the fork moves its sequences
        assert two.pos.tolist() == p.append(two.k_new[:, None], buf[:, None, 6:], [1] * 3)
        want = p.attend(two.q, 0.125, two.page_idx.tolist())
        tol, tol_lse = plain.bounds(BF16, 64, want[0], *want[2:])
        assert bool(((two.out.cpu().double() - want[0]).abs() <= tol).all())
        assert bool(((two.lse.cpu().double() - want[1]).abs() <= tol_lse + want[1].abs() * 2.0 ** -22).all())
        two.fork(parent)
        two.compact()
        assert p.fork([0, 0, 1], None)
        p.compact()
        for name in ("out", "lse", "pos", "page_idx", "done", "q"):
            assert same(getattr(one, name), getattr(two, name)), name
        for name in ("k_pages", "v_pages", "kmin", "kmax", "ctx_len", "table", "refs"):
            assert same(getattr(one.cache, name), getattr(two.cache, name)), name
        assert two.ctx_len.tolist() == p.ctx and torch.equal(two.cache.table.cpu(), p.table()) and two.done.item() == 1
    ops.pipeline_check()


def test_tables_and_lengths_of_64_bits_keep_their_values():
    """A number that 32 bits cannot hold stays what it is: a page that does not exist, a length above the capacity."""
    pair = Pair(2, 2, 1, 64, 16, 64, 8, summaries=False)
    pair.append([64, 20])
    table, lens = pair.cache.table.long().cpu(), pair.cache.ctx_len.long().cpu()
    for dev in ("cpu", "cuda"):
        odd, long = table.clone(), lens.clone()
        odd[0, 1] += 1 << 32
        odd[0, 2] = -(1 << 32) + 3
        long[1] = (1 << 32) + 20
        odd[1] = torch.tensor([4, 5, 6, 7])
        pair.cache.load(odd.to(dev), long.to(dev))
        with pytest.raises(L.SlsError, match="2 page-list entries"):
            ops.pipeline_check()
        held = pair.cache.table.cpu()
        assert not 0 <= held[0, 1] < 8 and not 0 <= held[0, 2] < 8 and held[0, [0, 3]].tolist() == table[0, [0, 3]].tolist()
        refs = [0] * 8
        for p in (int(table[0, 0]), int(table[0, 3]), 4, 5, 6, 7):  # all four pages: the length counts as the capacity
            refs[p] += 1
        assert pair.cache.refs.tolist() == refs
        with pytest.raises(ValueError, match="integers"):
            pair.cache.load(odd.bool().to(dev), lens.to(dev))
    pair.cache.load(table, lens)
    pair.check()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("batch,cap,lens", [(1, 32768, [1000]), (6, 8192, [8192, 1, 700, 4096, 17, 8000]),
                                            (40, 4096, [97 * i for i in range(1, 41)])])
def test_repeated_calls_give_equal_bits(dtype, batch, cap, lens):
    """In clusters and in ranges, dense and over lists, whatever ran in between."""
    pair = Pair(batch, 8, 2, 128, 16, cap, sum(-(-n // 16) for n in lens) + 4, dtype, summaries=False)
    gen = torch.Generator("cuda").manual_seed(7)
    kv = torch.randn((batch, max(lens), 4, 128), generator=gen, device="cuda").to(dtype)
    ops.paged_append(pair.desc, pair.cache, kv[:, :, :2], kv[:, :, 2:], new_len=ints(lens))
    q, other = (torch.randn((batch, 8, 128), generator=gen, device="cuda").to(dtype) for _ in range(2))
    idx = ints([pair.rng.permutation(cap // 16)[:60].tolist() for _ in range(2 * batch)])
    ws = ops.paged_attend_workspace(pair.desc, pair.cache)
    first = {}
    for turn in range(20):
        for name, lists in (("dense", None), ("lists", idx)):
            got = ops.paged_decode_attend(pair.desc, pair.cache, q, page_idx=lists, workspace=ws)
            ref = first.setdefault(name, got)
            assert same(got[0], ref[0]) and same(got[1], ref[1]), (name, turn)
            ops.paged_decode_attend(pair.desc, pair.cache, other, page_idx=lists, workspace=ws)
    ops.pipeline_check()
