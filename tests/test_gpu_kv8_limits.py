"""The 8-bit cache's calls at the limits of their kernels' tables: rows of more blocks than the choice keeps on chip, slices
of the longest list, KV heads that do not divide a cluster, and as many rows as the attend takes."""
import numpy as np
import pytest
import torch

from sparse_long_context_gb300 import ops
from tests.test_gpu_kv8 import Pair, attention, ints, query

pytestmark = pytest.mark.gpu


def filled(batch, hkv, d, block, nblk, lens, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    desc = ops.make_desc(batch, hkv, hkv, d, block, nblk * block, torch.bfloat16)
    cache = ops.Kv8Cache.empty(desc, "int8", block)
    for t in (cache.k_codes, cache.v_codes):
        t.random_(0, 256, generator=g)
    for t in (cache.k_scales, cache.v_scales):
        t.uniform_(generator=g)
    for t in (cache.k_tail, cache.v_tail):
        t.normal_(generator=g)
    mass = (torch.rand((batch, hkv, nblk), generator=g, device="cuda") * 500).floor()  # ties
    return desc, cache, mass, ints(lens)


def chosen(mass, n, keep, sinks, recent):
    """Kept blocks of every row, by a stable sort: the forced ones first, then by sum, ties to the lower block."""
    i = torch.arange(mass.shape[-1], device="cuda")
    key = mass.double().masked_fill((i < sinks) | (i >= n - recent), float("inf")).masked_fill(i >= n, -1.0)
    return torch.sort(torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :keep], dim=-1).values


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,hkv,d,nblk,keep", [(1, 2, 64, 9001, 5000), (1, 1, 128, 8192, 7), (2, 1, 64, 4097, 4096),
                                                   (38, 8, 64, 3100, 3001)])  # 304 rows: a CTA has 2048 entries of a list
def test_evict_from_long_rows(in_place, batch, hkv, d, nblk, keep):
    block = 16
    lens = [nblk * block - (b % 3) * 5 - (b // 3) * 16 for b in range(batch)]
    desc, cache, mass, ctx = filled(batch, hkv, d, block, nblk, lens, keep)
    names = ("k_codes", "v_codes", "k_scales", "v_scales")
    want = torch.stack([chosen(mass[b], lens[b] // block, keep, 2, 3) if lens[b] // block > keep else
                        torch.arange(keep, device="cuda").expand(hkv, -1) for b in range(batch)])
    assert min(n // block for n in lens) >= keep
    per = {n: getattr(cache, n).view(batch, hkv, nblk, -1) for n in names}
    ref = {n: torch.gather(x, 2, want[..., None].expand(-1, -1, -1, x.shape[-1])) for n, x in per.items()}
    ref_mass = torch.gather(mass, 2, want)
    tails = cache.k_tail.clone(), cache.v_tail.clone()
    if in_place:
        got, kept = ops.kv8_evict(desc, cache, ctx, mass, keep, 2, 3)
        to, sums = cache, mass
    else:
        desc2 = ops.make_desc(batch, hkv, hkv, d, block, (keep + 1) * block, torch.bfloat16)
        to = ops.Kv8Cache.empty(desc2, "int8", block)
        sums = torch.zeros((batch, hkv, keep + 1), device="cuda")
        got, kept = ops.kv8_evict(desc, cache, ctx, mass, keep, 2, 3, dst_desc=desc2, dst=to, mass_out=sums)
    assert got.tolist() == [keep * block + n % block for n in lens]
    assert torch.equal(kept.view(batch, hkv, keep).long(), want)
    for n in names:
        x = getattr(to, n)
        x = x.view(batch, hkv, x.shape[2] // (block if n.endswith("codes") else 1), -1)
        assert torch.equal(x[:, :, :keep], ref[n]), n
    assert torch.equal(sums[:, :, :keep], ref_mass)
    for b in range(batch):
        r = lens[b] % block
        assert torch.equal(to.k_tail[b, :, :r], tails[0][b, :, :r]) and torch.equal(to.v_tail[b, :, :r], tails[1][b, :, :r])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("hkv", [3, 5, 6, 7, 8, 9, 16, 19])
def test_single_tokens_of_many_heads(fmt, hkv):
    """A cluster of up to 8 CTAs per sequence takes the heads in turn; blocks are completed on the way."""
    p = Pair(2, hkv, hkv, 64 if hkv % 2 else 128, 64, fmt, 16, page=16, seed=hkv, meta=True)
    p.append([14, 31])
    for _ in range(4):
        p.append([1, 1])
    p.append([0, 1])
    p.check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("batch,hkv,cap", [(4096, 1, 64), (4096, 1, 1024), (1024, 4, 1024)])  # a CTA a row; ranges
def test_attend_of_as_many_rows_as_there_may_be(fmt, batch, hkv, cap):
    lens = np.random.default_rng(batch).integers(0, 40, batch).tolist()
    lens[-2], more = 0, [0] * batch
    more[7] = more[-1] = 60 if cap > 64 else 20  # two longer rows
    p = Pair(batch, 2 * hkv, hkv, 128, cap, fmt, 16, seed=cap)
    p.append(lens)
    p.append(more)
    attention(p, query(p, 1), mass_in=torch.rand_like(p.mass))
    pages = torch.arange(cap // 16, dtype=torch.int32, device="cuda").flip(0).expand(batch * hkv, -1).contiguous()
    attention(p, query(p, 2), pages=(pages, None))
