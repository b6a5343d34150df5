"""The paged cache on the GPU (append, selection, decode attention, fork, compaction) against the plain form of
tests/paged_plain.py."""
import math

import numpy as np
import pytest
import torch

from sparse_long_context_gb300 import _lib as L
from sparse_long_context_gb300 import ops
from tests import paged_plain as plain

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def same(a, b):
    return torch.equal(a.cpu().contiguous().view(torch.uint8), b.cpu().contiguous().view(torch.uint8))


class Pair:
    """A device cache and its plain form, changed together.  Pages begin with garbage (NaN among it), which stays where no
    token is written."""

    def __init__(self, batch, hq, hkv, d, page, cap, pool, dtype=BF16, summaries=True, seed=0):
        self.desc = ops.make_desc(batch, hq, hkv, d, page, cap, dtype)
        self.rng = np.random.default_rng(seed)
        self.dtype = dtype
        junk = lambda *s: torch.from_numpy(np.where(self.rng.random(s) < 0.2, np.nan, 1e4)).to(dtype)  # noqa: E731
        k, v = junk(pool, hkv, page, d), junk(pool, hkv, page, d)
        lo, hi = (junk(pool, hkv, d), junk(pool, hkv, d)) if summaries else (None, None)
        self.plain = plain.PlainPaged(batch, hkv, d, page, cap, k, v, lo, hi)
        self.cache = ops.PagedCache(self.desc, k.cuda(), v.cuda(), *((lo.cuda(), hi.cuda()) if summaries else ()))
        self.gain = np.exp(0.5 * self.rng.standard_normal(d))

    def new(self, shape, gain=1.0):
        return torch.from_numpy(self.rng.standard_normal(shape) * gain).to(self.dtype)

    def append(self, lens):
        d = self.desc
        t = max([*lens, 1])
        kv = torch.cat([self.new((d.batch, t, d.num_kv_heads, d.head_dim), self.gain),
                        self.new((d.batch, t, d.num_kv_heads, d.head_dim))], 2)  # one packed buffer: strided views
        dev = kv.cuda()
        pos = torch.full((d.batch,), 77, dtype=torch.int32, device="cuda")
        ops.paged_append(d, self.cache, dev[:, :, :d.num_kv_heads], dev[:, :, d.num_kv_heads:], new_len=ints(lens), pos_out=pos)
        want = self.plain.append(kv[:, :, :d.num_kv_heads], kv[:, :, d.num_kv_heads:], lens)
        assert pos.tolist() == want

    def fork(self, parent, keep=None):
        done = torch.full((1,), 7, dtype=torch.int32, device="cuda")
        ops.paged_fork(self.desc, self.cache, ints(parent), None if keep is None else ints(keep), done=done)
        ok = self.plain.fork(parent, keep)
        assert done.item() == int(ok)
        return ok

    def compact(self):
        moved = torch.full((self.cache.num_pages,), 7, dtype=torch.int32, device="cuda")
        ops.paged_compact(self.desc, self.cache, moved=moved)
        assert moved.tolist() == self.plain.compact()

    def check(self):
        p, c = self.plain, self.cache
        assert c.ctx_len.tolist() == p.ctx
        assert torch.equal(c.table.cpu(), p.table())
        assert c.refs.tolist() == p.refs()
        assert same(c.k_pages, p.k) and same(c.v_pages, p.v)
        if p.lo is not None:
            assert same(c.kmin, p.lo) and same(c.kmax, p.hi)
        ops.pipeline_check()

    def attend(self, q=None, pages=None, sink=None, **kw):
        d = self.desc
        q = self.new((d.batch, d.num_q_heads, d.head_dim)) if q is None else q
        out, lse = ops.paged_decode_attend(d, self.cache, q.cuda(), page_idx=None if pages is None else ints(pages),
                                           sink=None if sink is None else sink.cuda(), **kw)
        want = self.plain.attend(q, 1 / math.sqrt(d.head_dim), pages, sink)
        tol, tol_lse = plain.bounds(self.dtype, d.head_dim, want[0], *want[2:])
        out, lse = out.cpu().double(), lse.cpu().double()
        assert bool(((out - want[0]).abs() <= tol).all()), float(((out - want[0]).abs() / tol).max())
        dead = want[1].isinf()
        assert torch.equal(lse[dead], want[1][dead])
        assert bool(((lse - want[1])[~dead].abs() <= (tol_lse + want[1].abs() * 2.0 ** -22)[~dead]).all())
        ops.pipeline_check()
        return out


SHAPES = [(1, 1, 64, 16, BF16), (2, 4, 128, 16, BF16), (5, 3, 64, 32, F32), (3, 2, 128, 64, BF16), (7, 1, 128, 128, F32),
          (4, 8, 64, 256, BF16)]


@pytest.mark.parametrize("batch,hkv,d,page,dtype", SHAPES)
@pytest.mark.parametrize("summaries", [True, False])
def test_append_piece_by_piece(batch, hkv, d, page, dtype, summaries):
    pair = Pair(batch, hkv, hkv, d, page, 4 * page, batch * 4 + 3, dtype, summaries, seed=batch)
    pair.check()
    for step in range(7):
        lens = [int(pair.rng.integers(0, page + 2)) if (b + step) % 3 else 1 for b in range(batch)]
        pair.append(lens)
        pair.check()
    pair.append([2 * page - 1] * batch)  # some fit no more
    pair.check()


def test_append_counts_are_clamped_and_may_be_left_out():
    pair = Pair(3, 2, 2, 64, 16, 64, 12)
    kv = pair.new((3, 20, 2, 64))
    for lens in ([-5, 99, 0], [20, 20, 20], [20, 20, 20]):
        ops.paged_append(pair.desc, pair.cache, kv.cuda(), kv.cuda(), new_len=ints(lens))
        pair.plain.append(kv, kv, lens)
        pair.check()
    ops.paged_append(pair.desc, pair.cache, kv.cuda(), kv.cuda())  # every token of every sequence: 60 + 20 > 64 stays
    pair.plain.append(kv, kv, [20] * 3)
    pair.check()
    ops.paged_append(pair.desc, pair.cache, kv[:, :0].cuda(), kv[:, :0].cuda())
    pair.check()


def test_append_when_the_pool_runs_out():
    pair = Pair(6, 1, 1, 64, 16, 256, 9)
    pair.append([16, 5, 0, 16, 0, 3])
    pair.check()                      # 4 pages used, 5 free
    pair.append([40, 4, 33, 33, 1, 2])  # 3 + 0 + 3 (one too many) + 3 + 1 + 0
    pair.check()
    assert pair.plain.ctx == [56, 9, 0, 16, 0, 5]
    pair.append([0, 0, 17, 0, 1, 0])
    pair.check()
    pair.append([0, 7, 0, 0, 0, 1])
    pair.check()
    pair.append([1] * 6)
    pair.check()


def test_append_takes_the_lowest_free_pages():
    pair = Pair(40, 1, 1, 64, 16, 2048, 5000)
    pair.append([int(n) for n in pair.rng.integers(1, 2000, 40)])
    pair.fork([b if b % 3 else -1 for b in range(40)])
    pair.check()
    pair.append([0 if b % 3 else int(pair.rng.integers(1, 2048)) for b in range(40)])
    pair.check()


def test_append_to_a_shared_partial_page_of_a_callers_table_is_refused():
    pair = Pair(3, 1, 1, 64, 16, 64, 8)
    table = torch.full((3, 4), -1, dtype=torch.int32)
    table[0, 0] = table[1, 0] = 5
    table[2, 0] = 99
    pair.cache.load(table.cuda(), ints([3, 3, 4]))
    with pytest.raises(L.SlsError) as e:
        ops.pipeline_check()
    assert e.value.code == L.SLS_EDEVICE
    kv = pair.new((3, 1, 1, 64)).cuda()
    before = pair.cache.k_pages.clone()
    ops.paged_append(pair.desc, pair.cache, kv, kv)
    with pytest.raises(L.SlsError) as e:
        ops.pipeline_check()
    assert e.value.code == L.SLS_EDEVICE
    assert pair.cache.ctx_len.tolist() == [3, 3, 4] and same(pair.cache.k_pages, before)


@pytest.mark.parametrize("summaries", [True, False])
@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 64)])
def test_fork_shares_cuts_frees_and_reorders(dtype, d, summaries):
    pair = Pair(6, 2, 2, d, 16, 128, 40, dtype, summaries)
    pair.append([37, 16, 5, 64, 0, 1])
    pair.fork([0, 1, 0, 3, 0, 3], [99, 99, 20, 99, 37, 33])   # forks: a cut inside a page, a whole copy
    pair.check()
    pair.append([1, 1, 12, 17, 11, 15])
    pair.check()
    pair.fork([1, 0, 3, 2, 5, 4])                             # a permutation
    pair.check()
    pair.fork([0, 1, 2, 3, 4, 5], [0, 3, 16, 40, 1, 200])     # cuts in place
    pair.check()
    pair.append([3, 3, 3, 3, 3, 3])
    pair.check()
    pair.fork([3, 3, 3, 3, 3, 3], [17, 18, 32, 43, 43, 0])    # all of one
    pair.check()
    pair.fork([3, 3, 3, -1, -1, 5], [-4, 33, 33, 5, 5, 5])    # its pages pass to a lower user
    pair.check()
    pair.fork([-1] * 6)
    pair.check()
    assert pair.plain.refs() == [0] * 40
    pair.append([40] * 6)
    pair.check()


def test_fork_without_enough_pages_changes_nothing():
    pair = Pair(4, 1, 1, 64, 16, 128, 6)
    pair.append([40, 17, 0, 0])
    assert pair.plain.free() == [5]
    assert not pair.fork([0, -1, 0, 0])    # two copies, one page; sequence 1's pages come too late
    pair.check()
    assert not pair.fork([1, 1, 0, 0], [17, 3, 40, 40])
    pair.check()
    assert pair.fork([0, -1, 0, -1])
    pair.check()
    assert pair.fork([0, 0, 0, 0], [16, 32, 7, 39])
    pair.check()


def test_fork_counts_parents_that_do_not_exist():
    pair = Pair(3, 1, 1, 64, 16, 64, 9)
    pair.append([20, 3, 0])
    ops.paged_fork(pair.desc, pair.cache, ints([-2, 3, 1]), ints([1, 1, 1]))
    assert pair.plain.fork([-2, 3, 1], [1, 1, 1])
    with pytest.raises(L.SlsError) as e:
        ops.pipeline_check()
    assert e.value.code == L.SLS_EDEVICE
    pair.check()


@pytest.mark.parametrize("batch,hkv,d,page,dtype", SHAPES)
def test_random_runs_of_all_calls(batch, hkv, d, page, dtype):
    cap, g = 6 * page, 1 + batch % 4
    pair = Pair(batch, hkv * g, hkv, d, page, cap, batch * 4 + 2, dtype, seed=11 * batch + page)
    rng = pair.rng
    for step in range(24):
        what = rng.integers(0, 4)
        if what == 0:
            pair.append([int(n) for n in rng.integers(0, 2 * page, batch)])
        elif what == 1:
            pair.fork([int(p) for p in rng.integers(-1, batch, batch)], [int(n) for n in rng.integers(0, cap, batch)])
        elif what == 2:
            pair.fork([b if rng.random() < 0.7 else int(rng.integers(-1, batch)) for b in range(batch)])
        else:
            pair.compact()
        pair.check()
        if step % 6 == 5:
            pair.attend()


@pytest.mark.parametrize("batch,cap", [(5, 16 * 60000), (300, 16 * 1000), (1100, 64)])
def test_many_sequences_and_wide_tables(batch, cap):
    """Single tokens and forks of more sequences, and of wider tables, than one launch takes."""
    pair = Pair(batch, 1, 1, 64, 16, cap, 3 * batch + 40)
    rng = pair.rng
    for step in range(3):
        pair.append([int(n) for n in rng.integers(0, 2, batch)])
        pair.append([int(n) for n in rng.integers(0, 20, batch)])
        kv = pair.new((batch, 1, 1, 64))
        ops.paged_append(pair.desc, pair.cache, kv.cuda(), kv.cuda())
        pair.plain.append(kv, kv, [1] * batch)
        pair.check()
        pair.fork([b if rng.random() < 0.5 else int(rng.integers(-1, batch)) for b in range(batch)],
                  [int(n) for n in rng.integers(0, 40, batch)])
        pair.check()
    for _ in range(4):  # some of them for want of pages
        pair.fork([int(rng.integers(0, batch)) for _ in range(batch)], [31] * batch)
        pair.check()
        pair.append([int(n) for n in rng.integers(0, 60, batch)])
        pair.check()


@pytest.mark.parametrize("pool,cap", [(31, 128), (32, 128), (33, 128), (1000, 2048), (40000, 65536)])
def test_compact_pools_of_many_sizes(pool, cap):
    pair = Pair(12, 1, 1, 64, 16, cap, pool, summaries=pool < 2000)
    pair.compact()  # nothing to move
    pair.check()
    pair.append([min(int(n), pool // 13 * 16) for n in pair.rng.integers(1, cap, 12)])
    pair.fork([b if b % 2 else -1 for b in range(12)])
    pair.compact()
    pair.check()
    pair.append([5] * 12)
    pair.check()
    pair.compact()
    pair.check()
    pair.append([cap // 4] * 12)
    pair.compact()
    pair.check()


def test_compact_of_a_full_pool():
    pair = Pair(2, 1, 1, 64, 16, 512, 32)
    pair.append([256, 250])
    assert not pair.plain.free()
    pair.compact()
    pair.check()


@pytest.mark.parametrize("g", [1, 3, 8])
@pytest.mark.parametrize("batch,hkv,d,page,dtype", SHAPES)
def test_attend_lengths(batch, hkv, d, page, dtype, g):
    cap = 8 * page
    pair = Pair(batch, hkv * g, hkv, d, page, cap, batch * 8, dtype, summaries=False, seed=g)
    q = pair.new((batch, hkv * g, d), 2.0)
    pair.attend(q)  # no token: zeros, lse -inf
    pair.attend(q, sink=torch.randn(hkv * g))
    some = [1, 15, 16, 17, page - 1, page, page + 1, 3 * page + 7, cap]
    pair.append([some[(b + g) % 9] for b in range(batch)])
    pair.attend(q)
    pair.attend(q, sink=torch.randn(hkv * g))
    pair.append([some[(b + g + 4) % 5] for b in range(batch)])
    pair.attend(q)


@pytest.mark.parametrize("batch,hkv,d,page,dtype", SHAPES)
def test_attend_lists(batch, hkv, d, page, dtype):
    g = 1 + batch % 5
    pair = Pair(batch, hkv * g, hkv, d, page, 16 * page, batch * 16, dtype, summaries=False)
    pair.append([int(n) for n in pair.rng.integers(1, 16 * page, batch)])
    rows = batch * hkv
    for width in (1, 5, 16):
        lists = pair.rng.integers(0, 16, (rows, width))
        for r in range(rows):  # distinct pages, in any order, with gaps; some past the context
            lists[r] = pair.rng.permutation(16)[:width]
            lists[r][pair.rng.random(width) < 0.2] = -1
        lists = lists.tolist()
        lists[0] = [-1] * width
        q = pair.new((batch, hkv * g, d), 2.0)
        pair.attend(q, lists, torch.randn(hkv * g))
        a = pair.attend(q, lists)
        # count and k_fixed cut the lists
        count = [int(n) for n in pair.rng.integers(-1, width + 3, rows)]
        out, _ = ops.paged_decode_attend(pair.desc, pair.cache, q.cuda(), page_idx=ints(lists), count=ints(count))
        cut, _ = ops.paged_decode_attend(pair.desc, pair.cache, q.cuda(), page_idx=ints(
            [x[:max(n, 0)] + [-1] * (width - max(min(n, width), 0)) for x, n in zip(lists, count)]))
        assert bool(((out - cut).abs() <= 2.0 ** -7 * cut.abs() + 1e-2).all())
        out, _ = ops.paged_decode_attend(pair.desc, pair.cache, q.cuda(), page_idx=ints(lists), k_fixed=0)
        assert not out.any() and a.shape == out.shape


def test_attend_skips_and_counts_bad_entries():
    pair = Pair(2, 4, 2, 128, 16, 256, 40, summaries=False)
    pair.append([200, 130])
    q = pair.new((2, 4, 128))
    lists = [[0, 3, 5], [1, 2, -1], [4, 6, 7], [8, 0, 2]]
    good, _ = ops.paged_decode_attend(pair.desc, pair.cache, q.cuda(), page_idx=ints([[0, 3, -1], [-1, 2, -1], [4, 6, 7], [8, -1, 2]]))
    ops.pipeline_check()
    lists[0][2], lists[1][0], lists[3][1] = 16, -2, 1 << 30
    out, _ = ops.paged_decode_attend(pair.desc, pair.cache, q.cuda(), page_idx=ints(lists))
    with pytest.raises(L.SlsError, match="3 page-list entries"):
        ops.pipeline_check()
    assert same(out, good)
    # a table with holes: their tokens are missing
    pair.cache.table[0, 5], pair.cache.table[1, 0] = 40, -7
    out, lse = ops.paged_decode_attend(pair.desc, pair.cache, q.cuda())
    with pytest.raises(L.SlsError) as e:
        ops.pipeline_check()
    assert e.value.code == L.SLS_EDEVICE
    want = ops.paged_decode_attend(pair.desc, pair.cache, q.cuda(), page_idx=ints(
        [[p for p in range(16) if p != 5] + [-1]] * 2 + [[p for p in range(1, 16)] + [-1]] * 2))[0]
    assert bool(((out - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -10).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_rows_of_many_lengths(dtype):
    """Ranges over all rows and clusters, by the capacity; rows from none to thousands of tokens."""
    for batch, hkv, g, cap in ((30, 5, 2, 2048), (3, 1, 8, 16384), (150, 2, 1, 512)):
        pair = Pair(batch, hkv * g, hkv, 64, 16, cap, batch * cap // 32, dtype, summaries=False)
        lens = np.minimum(pair.rng.exponential(cap / 6, batch), cap).astype(int)
        lens[::7] = 0
        pair.append([int(n) for n in lens])
        pair.attend(pair.new((batch, hkv * g, 64), 2.0), sink=torch.randn(hkv * g) if batch == 30 else None)


def test_attend_repeats_bit_for_bit_on_any_stream_and_in_graphs():
    pair = Pair(9, 12, 2, 128, 16, 8192, 4700, summaries=False)
    pair.append([int(n) for n in pair.rng.integers(1, 8192, 9)])
    q = pair.new((9, 12, 128)).cuda()
    ws = ops.paged_attend_workspace(pair.desc, pair.cache)
    first = ops.paged_decode_attend(pair.desc, pair.cache, q, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = ops.paged_decode_attend(pair.desc, pair.cache, q, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert same(first[0], again[0]) and same(first[1], again[1])
    graph = torch.cuda.CUDAGraph()
    out, lse = torch.zeros_like(q), torch.zeros(9, 12, device="cuda")
    with torch.cuda.graph(graph):
        ops.paged_decode_attend(pair.desc, pair.cache, q, out=out, lse=lse, workspace=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert same(first[0], out) and same(first[1], lse)


@pytest.mark.parametrize("dtype,d,page,k", [(BF16, 128, 16, 20), (BF16, 64, 32, 7), (F32, 64, 16, 33), (F32, 128, 64, 3)])
def test_select_finds_what_the_row_selection_finds(dtype, d, page, k):
    batch, hkv, g, cap = 5, 2, 3, 128 * page
    pair = Pair(batch, hkv * g, hkv, d, page, cap, 700, dtype)
    pair.append([int(n) for n in pair.rng.integers(1, cap, batch)])
    pair.check()
    q = pair.new((batch, hkv * g, d))
    at = pair.cache.table.clamp(min=0).long()
    rows = lambda x: x[at].transpose(1, 2).contiguous()  # noqa: E731  [B, Hkv, Cap/P, D]
    for first, last in ((0, 0), (1, page), (2, 0)):
        want = ops.select_pages(pair.desc, q.cuda(), rows(pair.cache.kmin), rows(pair.cache.kmax), pair.cache.ctx_len, k, first, last)
        got = ops.paged_select_pages(pair.desc, pair.cache, q.cuda(), k, first, last)
        assert torch.equal(want, got)
        ops.pipeline_check()
    pair.attend(q, got.tolist())


@pytest.mark.parametrize("dtype,hkv,batch,cap", [(BF16, 3, 60, 2048), (F32, 4, 90, 1024), (BF16, 8, 25, 16 * 4096), (BF16, 2, 80, 16 * 4200),
                                                 (F32, 1, 2, 16 * 4097)])
def test_select_of_more_rows_than_sms_and_of_the_widest_rows(dtype, hkv, batch, cap):
    pair = Pair(batch, 4 * hkv, hkv, 64, 16, cap, 9000, dtype)
    lens = [int(n) for n in pair.rng.integers(1, min(cap, 9000 // batch * 16 - 16), batch)]
    pair.append(lens[:-1] + [min(cap, 8000)])
    q = pair.new((batch, 4 * hkv, 64)).cuda()
    at = pair.cache.table.clamp(min=0).long()
    lo, hi = (x[at].transpose(1, 2).contiguous() for x in (pair.cache.kmin, pair.cache.kmax))
    for k, first, last in ((20, 1, 64), (63, 0, 0)):
        assert torch.equal(ops.paged_select_pages(pair.desc, pair.cache, q, k, first, last),
                           ops.select_pages(pair.desc, q, lo, hi, pair.cache.ctx_len, k, first, last))
    ops.pipeline_check()


@pytest.mark.parametrize("batch", [3, 100])
@pytest.mark.parametrize("dtype,flags", [(F32, {}), (BF16, dict(cuda_cores=True)), (BF16, {})])
@pytest.mark.parametrize("g", [1, 2, 4, 7])
def test_select_group_sizes_and_kernels(g, dtype, flags, batch):
    """Every scorer, in one launch (few rows) and in two (many rows, or the CUDA-core flag)."""
    for d in (64, 128):
        pair = Pair(batch, 2 * g, 2, d, 16, 1024, 1500, dtype)
        pair.append([int(n) for n in pair.rng.integers(1, 240 if batch > 9 else 1024, batch)])
        desc = ops.make_desc(batch, 2 * g, 2, d, 16, 1024, dtype, **flags)
        q = pair.new((batch, 2 * g, d)).cuda()
        at = pair.cache.table.clamp(min=0).long()
        lo, hi = (x[at].transpose(1, 2).contiguous() for x in (pair.cache.kmin, pair.cache.kmax))
        for k, first, last in ((6, 1, 17), (11, 0, 0)):
            assert torch.equal(ops.paged_select_pages(desc, pair.cache, q, k, first, last),
                               ops.select_pages(desc, q, lo, hi, pair.cache.ctx_len, k, first, last))
    ops.pipeline_check()


def test_select_counts_bad_entries_and_scores_them_as_zeros():
    pair = Pair(2, 4, 2, 64, 16, 1024, 130)
    pair.append([1000, 640])
    q = pair.new((2, 4, 64)).cuda()
    at = pair.cache.table.clamp(min=0).long()
    lo, hi = (x[at].transpose(1, 2).contiguous() for x in (pair.cache.kmin, pair.cache.kmax))
    pair.cache.table[0, 7], pair.cache.table[0, 9], pair.cache.table[1, 30] = -1, 130, 1 << 30
    for b, p in ((0, 7), (0, 9), (1, 30)):
        lo[b, :, p] = hi[b, :, p] = 0
    got = ops.paged_select_pages(pair.desc, pair.cache, q, 12, 1, 20)
    with pytest.raises(L.SlsError, match="6 page-list entries"):  # for each of the two KV heads
        ops.pipeline_check()
    assert torch.equal(got, ops.select_pages(pair.desc, q, lo, hi, pair.cache.ctx_len, 12, 1, 20))


@pytest.mark.parametrize("pool", [1, 2, 3])
def test_pools_of_a_few_pages(pool):
    pair = Pair(3, 2, 1, 64, 16, 64, pool)
    pair.append([5, 16, 1])
    pair.check()
    pair.attend()
    pair.fork([1, 0, 2])
    pair.check()
    pair.fork([0, 0, 0], [3, 5, 1])
    pair.check()
    pair.fork([-1, 1, 2])
    pair.compact()
    pair.check()
    pair.append([1, 1, 1])
    pair.check()
    pair.attend()


@pytest.mark.parametrize("batch,hkv,cap,dtype", [(1, 1, 2048, BF16), (2, 3, 16 * 700, BF16), (40, 2, 16 * 130, BF16), (77, 1, 1024, F32),
                                                 (90, 2, 1024, BF16), (3, 1, 16 * 2500, F32)])
def test_select_clusters_ties_and_few_pages(batch, hkv, cap, dtype):
    """One CTA or several a row, or two launches; scores that are equal; rows of no more pages than the budget."""
    pair = Pair(batch, hkv * 2, hkv, 64, 16, cap, min(batch * cap // 16, 6000), dtype)
    lens = [int(n) for n in pair.rng.integers(1, min(cap, 6000 // batch * 16), batch)]
    lens[0], lens[-1] = 17, lens[-1]
    pair.append(lens)
    q = torch.round(pair.new((batch, hkv * 2, 64)) * 2) / 2
    # summaries of few values: many equal scores
    pair.cache.kmin.copy_(torch.round(pair.new(pair.cache.kmin.shape)).clamp(-1, 0))
    pair.cache.kmax.copy_(torch.round(pair.new(pair.cache.kmin.shape)).clamp(0, 1))
    at = pair.cache.table.clamp(min=0).long()
    rows = lambda x: x[at].transpose(1, 2).contiguous()  # noqa: E731
    lo, hi = rows(pair.cache.kmin), rows(pair.cache.kmax)
    x = torch.einsum("bhgd,bhpd->bhgp", q.cuda().view(batch, hkv, 2, 64).double().clamp(min=0), hi.double()) + torch.einsum(
        "bhgd,bhpd->bhgp", q.cuda().view(batch, hkv, 2, 64).double().clamp(max=0), lo.double())
    x = x.amax(2).cpu()
    for k, first, last in ((1, 0, 0), (5, 1, 16), (33, 0, 40), (64, 3, 100)):
        got = ops.paged_select_pages(pair.desc, pair.cache, q.cuda(), k, first, last)
        assert torch.equal(got, ops.select_pages(pair.desc, q.cuda(), lo, hi, pair.cache.ctx_len, k, first, last))
        got = got.view(batch, hkv, k).tolist()
        for b in range(batch):
            n = -(-lens[b] // 16)
            for j in range(hkv):
                must = {p for p in range(n) if p < first or (last and p >= max(lens[b] - last, 0) // 16)}
                others = sorted((p for p in range(n) if p not in must), key=lambda p: (-float(x[b, j, p]), p))
                want = sorted([*must, *others[:max(k - len(must), 0)]])
                assert got[b][j] == want + [-1] * (k - len(want)), (b, j)


def test_select_of_rows_wider_than_one_cta():
    cap = 16 * 9000
    pair = Pair(1, 2, 1, 64, 16, cap, 9000, summaries=True)
    pair.append([cap - 5])
    q = pair.new((1, 2, 64)).cuda()
    at = pair.cache.table.clamp(min=0).long()
    rows = lambda x: x[at].transpose(1, 2).contiguous()  # noqa: E731
    want = ops.select_pages(pair.desc, q, rows(pair.cache.kmin), rows(pair.cache.kmax), pair.cache.ctx_len, 100, 1, 64)
    assert torch.equal(want, ops.paged_select_pages(pair.desc, pair.cache, q, 100, 1, 64))


def test_attend_wait_that_gives_up_is_reported():
    desc = ops.make_desc(2, 4, 2, 128, 16, 256, BF16, test_wait_timeout=True)
    pair = Pair(2, 4, 2, 128, 16, 256, 40, summaries=False)
    pair.append([200, 130])
    q = pair.new((2, 4, 128)).cuda()
    out, lse = ops.paged_decode_attend(desc, pair.cache, q)
    with pytest.raises(L.SlsError) as e:
        ops.pipeline_check()
    assert e.value.code == L.SLS_ETIMEOUT
    assert out[0, :2].isnan().all() and not out[1].isnan().any()
    pair.attend(q.cpu())


def test_attend_refuses_lists_without_entries():
    pair = Pair(2, 4, 2, 128, 16, 256, 40, summaries=False)
    pair.append([200, 130])
    q = pair.new((2, 4, 128)).cuda()
    with pytest.raises(ValueError, match="page_idx"):
        ops.paged_decode_attend(pair.desc, pair.cache, q, page_idx=torch.empty((4, 0), dtype=torch.int32, device="cuda"))
    pair.attend(q.cpu(), pages=[[-1]] * 4)  # a list that holds nothing


def test_load_refuses_before_it_changes_anything():
    pair = Pair(2, 4, 2, 128, 16, 256, 40, summaries=False)
    pair.append([200, 130])
    table, lens = pair.cache.table.clone(), pair.cache.ctx_len.clone()
    for t, n in ((table[0], lens), (table[:1], lens), (table, lens[:1]), (table, lens[0]), (table.float(), lens)):
        with pytest.raises(ValueError):
            pair.cache.load(t, n)
        pair.check()
    pair.cache.load(table.cpu().long(), lens.cpu().long())
    pair.check()


# the first sequence empty (a row's cluster); a first range that is moved to the start of the second one
@pytest.mark.parametrize("cap,lens", [(256, [0, 200, 130]), (65536, [1504] + [88] * 99)])
def test_attend_wait_that_gives_up_is_that_of_the_first_tokens(cap, lens):
    desc = ops.make_desc(len(lens), 2, 1, 128, 16, cap, BF16, test_wait_timeout=True)
    pair = Pair(len(lens), 2, 1, 128, 16, cap, 1000, summaries=False)
    pair.append(lens)
    q = pair.new((len(lens), 2, 128)).cuda()
    out, _ = ops.paged_decode_attend(desc, pair.cache, q)
    with pytest.raises(L.SlsError) as e:
        ops.pipeline_check()
    assert e.value.code == L.SLS_ETIMEOUT
    first = next(i for i, n in enumerate(lens) if n)
    assert out[first].isnan().all() and not out[:first].isnan().any() and not out[first + 1:].isnan().any()
    pair.attend(q.cpu())
