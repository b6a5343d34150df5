"""Page selection over summaries and queries that are not finite, by every scorer (bf16 on the tensor cores, the CUDA cores, fp32;
row caches in both top-k kernels, one-token pages, pools in one launch and in two, the one-launch step) against the definition in 64
bits: a channel adds q kmax where q > 0, q kmin where q < 0 and nothing where q is zero or NaN; a page one of whose heads has
no score (infinities of both signs, a NaN summary) ranks above every score and below the forced pages, ties to the lower page."""
import math

import pytest
import torch

from sparse_long_context_gb300 import ops

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
KINDS = ["unused_sides", "every_page_without_a_score", "mixed", "queries"]


def make(kind, batch, hkv, g, d, pages, dtype, seed):
    """q [B, Hkv, G, D] and summaries [B, Hkv, NP, D] of small whole and half numbers (every sum is exact), with the
    values of `kind` among them."""
    gen = torch.Generator().manual_seed(seed)
    q = torch.randint(-4, 5, (batch, hkv, g, d), generator=gen).double() / 2
    lo = torch.randint(-6, 3, (batch, hkv, pages, d), generator=gen).double()
    hi = lo + torch.randint(0, 5, lo.shape, generator=gen).double()
    at = lambda share: torch.rand(lo.shape[:3], generator=gen) < share  # noqa: E731
    if kind == "unused_sides":  # infinities that no head's bound takes: the scores are finite
        q[..., 3] = -q[..., 3].abs() - 1   # takes kmin
        q[..., 5] = q[..., 5].abs() + 1    # takes kmax
        q[..., 6] = 0.0
        hi[..., 3] = math.inf
        lo[..., 5][at(0.5)] = -math.inf
        lo[..., 6], hi[..., 6] = -math.inf, math.inf
    elif kind == "every_page_without_a_score":  # +inf and -inf in one sum
        q[..., 1] = q[..., 1].abs() + 1
        q[..., 2] = q[..., 2].abs() + 1
        hi[..., 1] = math.inf
        lo[..., 2] = hi[..., 2] = -math.inf
    elif kind == "mixed":
        q[..., 0] = q[..., 0].abs() + 1
        hi[..., 0][at(0.02)] = math.inf                      # scores of +inf
        few = at(0.02)
        lo[..., 0][few] = hi[..., 0][few] = -math.inf        # of -inf
        hi[..., 7][at(0.01)] = math.nan                      # none for heads with q > 0 there
        lo[..., 8][at(0.01)] = math.nan
        wide = at(0.3)
        lo[..., 9][wide], hi[..., 9][wide] = -math.inf, math.inf
    else:  # queries: an infinite one, a NaN
        q[0, :, 0, 4] = math.inf
        q[:, :, -1, 11] = math.nan
        lo[..., 4], hi[..., 4] = lo[..., 4].clamp(max=-1), hi[..., 4].clamp(min=0)
    return q.to(dtype), lo.to(dtype), hi.to(dtype)


def lists(q, lo, hi, lens, page, k, first, last):
    """What has to be selected: [B * Hkv, k]."""
    q, lo, hi = (x.double()[:, :, None] if i else x.double()[:, :, :, None] for i, x in enumerate((q, lo, hi)))
    term = torch.where(q > 0, q * hi, torch.where(q < 0, q * lo, torch.zeros((), dtype=torch.float64)))
    head = term.sum(-1)                                                 # [B, Hkv, G, NP]
    none = head.isnan().any(2)
    score = head.masked_fill(head.isnan(), -math.inf).amax(2)
    rows = []
    for b in range(q.shape[0]):
        n = -(-lens[b] // page)
        must = {p for p in range(n) if p < first or (last and p >= max(lens[b] - last, 0) // page)}
        for h in range(q.shape[1]):
            if n <= k:
                rows.append(list(range(n)) + [-1] * (k - n))
                continue
            s, bad = score[b, h].tolist(), none[b, h].tolist()
            others = sorted((p for p in range(n) if p not in must), key=lambda p: (not bad[p], -s[p] if not bad[p] else 0.0, p))
            rows.append(sorted([*must, *others[:k - len(must)]]))
    return torch.tensor(rows, dtype=torch.int32)


SCORERS = [(BF16, {}), (BF16, dict(cuda_cores=True)), (F32, {})]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("g,d", [(1, 64), (2, 128), (3, 64), (4, 128), (7, 128), (8, 64)])
@pytest.mark.parametrize("dtype,flags", SCORERS)
def test_rows(dtype, flags, g, d, kind):
    batch, hkv, page, cap = 2, 2, 16, 16 * 300
    q, lo, hi = make(kind, batch, hkv, g, d, 300, dtype, 10 * g + d)
    lens = [cap, 4001]
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    desc = ops.make_desc(batch, hkv * g, hkv, d, page, cap, dtype, **flags)
    qd = q.reshape(batch, hkv * g, d).cuda()
    for k, first, last in ((20, 1, 40), (33, 0, 0), (5, 2, 16)):
        got = ops.select_pages(desc, qd, lo.cuda(), hi.cuda(), ctx, k, first, last)
        assert torch.equal(got.cpu(), lists(q, lo, hi, lens, page, k, first, last)), (k, first, last)
    ops.pipeline_check()


@pytest.mark.parametrize("kind", ["unused_sides", "mixed"])
@pytest.mark.parametrize("dtype,flags", SCORERS)
def test_wide_rows(dtype, flags, kind):
    """More pages than one top-k CTA holds: the scoring CTAs send candidates."""
    pages, g, d = 9000, 3, 64
    q, lo, hi = make(kind, 1, 1, g, d, pages, dtype, 5)
    lens = [16 * pages - 3]
    desc = ops.make_desc(1, g, 1, d, 16, 16 * pages, dtype, **flags)
    got = ops.select_pages(desc, q.reshape(1, g, d).cuda(), lo.cuda(), hi.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                           200, 1, 64)
    assert torch.equal(got.cpu(), lists(q, lo, hi, lens, 16, 200, 1, 64))


@pytest.mark.parametrize("kind", ["mixed", "queries"])
@pytest.mark.parametrize("dtype,flags", SCORERS)
def test_one_token_pages(dtype, flags, kind):
    q, lo, _ = make(kind, 2, 2, 3, 64, 500, dtype, 3)
    lens = [500, 333]
    desc = ops.make_desc(2, 6, 2, 64, 1, 500, dtype, **flags)
    keys = lo.cuda()
    got = ops.select_pages(desc, q.reshape(2, 6, 64).cuda(), keys, keys, torch.tensor(lens, dtype=torch.int32, device="cuda"), 40, 1, 7)
    assert torch.equal(got.cpu(), lists(q, lo, lo, lens, 1, 40, 1, 7))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("g,d", [(1, 64), (3, 128), (8, 128), (6, 64)])
def test_the_one_launch_step(g, d, kind):
    batch, hkv, page, cap = 2, 2, 16, 16 * 300
    q, lo, hi = make(kind, batch, hkv, g, d, 300, BF16, 7 * g + d)
    lens = [cap, 4001]
    desc = ops.make_desc(batch, hkv * g, hkv, d, page, cap, BF16)
    kv = torch.zeros((batch, hkv, cap, d), dtype=BF16, device="cuda")
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    assert ops.quest_step_splits(desc, 20) > 0
    idx = torch.empty((batch * hkv, 20), dtype=torch.int32, device="cuda")
    ops.quest_decode_step(desc, q.reshape(batch, hkv * g, d).cuda(), kv, kv, lo.cuda(), hi.cuda(), ctx, 20, 1, 40, page_idx=idx)
    assert torch.equal(idx.cpu(), lists(q, lo, hi, lens, page, 20, 1, 40))
    ops.pipeline_check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("batch,pages", [(2, 300), (90, 100), (1, 9000)])  # a cluster a row; a CTA a row; two launches
@pytest.mark.parametrize("dtype,flags,g,d", [(BF16, {}, 1, 64), (BF16, {}, 5, 128), (BF16, dict(cuda_cores=True), 3, 64), (F32, {}, 4, 64),
                                             (F32, {}, 7, 128)])
def test_pools(dtype, flags, g, d, batch, pages, kind):
    hkv, cap = 2, 16 * pages
    q, lo, hi = make(kind, batch, hkv, g, d, pages, dtype, batch + g)
    lens = [cap - 37 * (b % 7) for b in range(batch)]
    pool = batch * pages
    ids = torch.randperm(pool, generator=torch.Generator().manual_seed(1))
    table = ids.view(batch, pages).to(torch.int32)
    desc = ops.make_desc(batch, hkv * g, hkv, d, 16, cap, dtype, **flags)
    kmin, kmax = torch.empty((pool, hkv, d), dtype=dtype), torch.empty((pool, hkv, d), dtype=dtype)
    kmin[table.long().view(-1)] = lo.transpose(1, 2).reshape(pool, hkv, d)
    kmax[table.long().view(-1)] = hi.transpose(1, 2).reshape(pool, hkv, d)
    kv = torch.zeros((pool, hkv, 16, d), dtype=dtype, device="cuda")
    cache = ops.PagedCache(desc, kv, kv.clone(), kmin.cuda(), kmax.cuda())
    cache.load(table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    got = ops.paged_select_pages(desc, cache, q.reshape(batch, hkv * g, d).cuda(), 20, 1, 40)
    assert torch.equal(got.cpu(), lists(q, lo, hi, lens, 16, 20, 1, 40))
    ops.pipeline_check()


@pytest.mark.parametrize("dtype,flags", SCORERS)
@pytest.mark.parametrize("batch", [2, 90])
def test_pages_missing_from_a_table_beside_an_infinite_query(dtype, flags, batch):
    """A missing page scores as a summary of zeros; with an infinite query that is no number, and no memory is read for it."""
    q, lo, hi = make("queries", batch, 1, 2, 64, 100, dtype, 4)
    lens = [1600] * batch
    table = torch.arange(batch * 100, dtype=torch.int32).view(batch, 100)
    desc = ops.make_desc(batch, 2, 1, 64, 16, 1600, dtype, **flags)
    kv = torch.zeros((batch * 100, 1, 16, 64), dtype=dtype, device="cuda")
    cache = ops.PagedCache(desc, kv, kv.clone(), lo.reshape(-1, 1, 64).cuda(), hi.reshape(-1, 1, 64).cuda())
    cache.load(table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    cache.table[0, 50], cache.table[0, 51] = -1, 1 << 30
    lo[0, 0, 50:52] = hi[0, 0, 50:52] = 0
    got = ops.paged_select_pages(desc, cache, q.reshape(batch, 2, 64).cuda(), 20, 1, 40)
    with pytest.raises(ops.L.SlsError, match="2 page-list entries"):
        ops.pipeline_check()
    assert torch.equal(got.cpu(), lists(q, lo, hi, lens, 16, 20, 1, 40))
