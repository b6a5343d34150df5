"""The 8-bit cache on the GPU (append, decode attention, eviction and the step built of them) against the plain 64-bit
forms of tests/kv8_plain.py."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from sparse_long_context_gb300 import _lib as L
from sparse_long_context_gb300 import harness, ops
from tests import kv8_plain as plain

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def bf16(rng, shape, gain=1.0):
    x = rng.standard_normal(shape) * gain
    return torch.from_numpy(x).to(torch.bfloat16)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def same(a, b):
    return torch.equal(a.reshape(-1).view(torch.uint8), b.reshape(-1).view(torch.uint8))


class Pair:
    """A device cache and its plain rows, appended together."""

    def __init__(self, batch, hq, hkv, d, cap, fmt, block, page=16, seed=0, meta=False):
        self.desc = ops.make_desc(batch, hq, hkv, d, page, cap, torch.bfloat16)
        self.cache = ops.Kv8Cache.empty(self.desc, fmt, block)
        self.ctx = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.rows = [[plain.PlainCache(fmt, block, d) for _ in range(hkv)] for _ in range(batch)]
        self.rng = np.random.default_rng(seed)
        self.gain = np.exp(0.5 * self.rng.standard_normal(d))
        self.keys = [[[] for _ in range(hkv)] for _ in range(batch)]
        self.kmin = self.kmax = None
        if meta:
            self.kmin = torch.zeros((batch, hkv, cap // page, d), dtype=torch.bfloat16, device="cuda")
            self.kmax = torch.zeros_like(self.kmin)
        self.mass = torch.full((batch, hkv, cap // block), 7.0, device="cuda")

    def append(self, lens, edit=None):
        d = self.desc
        t = max(lens)
        kv = torch.cat([bf16(self.rng, (d.batch, t, d.num_kv_heads, d.head_dim), self.gain),
                        bf16(self.rng, (d.batch, t, d.num_kv_heads, d.head_dim))], 2)  # one packed buffer: strided views
        if edit:
            edit(kv)
        dev = kv.cuda()
        pos = torch.zeros_like(self.ctx)
        before = self.ctx.tolist()
        ops.kv8_append(d, self.cache, dev[:, :, :d.num_kv_heads], dev[:, :, d.num_kv_heads:], self.ctx, new_len=ints(lens),
                       kmin=self.kmin, kmax=self.kmax, mass=self.mass, pos_out=pos)
        x = kv.double().numpy()
        for b, n in enumerate(lens):
            n = max(0, min(n, t))
            if before[b] + n > d.capacity:
                n = 0
            assert int(pos[b]) == (before[b] if n else -1)
            for h in range(d.num_kv_heads):
                self.rows[b][h].append(x[b, :n, h], x[b, :n, d.num_kv_heads + h])
                self.keys[b][h].extend(x[b, :n, h])

    def check(self):
        d, c = self.desc, self.cache
        kc, vc = c.k_codes.cpu().numpy(), c.v_codes.cpu().numpy()
        ks, vs = c.k_scales.cpu().numpy(), c.v_scales.cpu().numpy()
        kt, vt = c.k_tail.double().cpu().numpy(), c.v_tail.double().cpu().numpy()
        mass = self.mass.cpu().numpy()
        for b in range(d.batch):
            for h in range(d.num_kv_heads):
                row = self.rows[b][h]
                assert int(self.ctx[b]) == len(row)
                for j, (a, s, a2, s2) in enumerate(row.blocks):
                    at = slice(j * c.block, (j + 1) * c.block)
                    assert (plain.value(kc[b, h, at], c.fmt) == plain.value(a, c.fmt)).all()
                    assert (plain.value(vc[b, h, at], c.fmt) == plain.value(a2, c.fmt)).all()
                    np.testing.assert_array_equal(ks[b, h, j], s)   # one IEEE division
                    np.testing.assert_array_equal(vs[b, h, j], s2)
                n = len(row.blocks)
                assert (mass[b, h, :n] == 0).all() and (mass[b, h, n:] == 7).all()
                assert (kc[b, h, n * c.block:] == 0).all() and (ks[b, h, n:] == 0).all()  # untouched
                for t, (k, v) in enumerate(zip(row.tail_k, row.tail_v)):
                    np.testing.assert_array_equal(kt[b, h, t], k)
                    np.testing.assert_array_equal(vt[b, h, t], v)
                if self.kmin is not None:
                    p = d.page_size
                    for g in range(0, len(self.keys[b][h]), p):
                        keys = np.array(self.keys[b][h][g:g + p])
                        assert (self.kmin[b, h, g // p].double().cpu().numpy() == keys.min(0)).all()
                        assert (self.kmax[b, h, g // p].double().cpu().numpy() == keys.max(0)).all()


CHUNKS = [[33, 1, 0], [1, 1, 1], [70, 15, 16], [1, 129, 5], [0, 47, 31], [1, 1, 1], [95, 3, 64], [1, 1, 1]]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("d,block,page,meta", [(128, 64, 16, True), (64, 16, 64, True), (128, 32, 32, True), (64, 256, 4, True),
                                               (128, 128, 256, True), (128, 16, 16, False)])
def test_append_in_chunks(fmt, d, block, page, meta):
    p = Pair(3, 2, 2, d, 512, fmt, block, page, seed=d + block, meta=meta)
    for lens in CHUNKS:
        p.append(lens)
        p.check()


def test_append_token_by_token_equals_one_chunk():
    a, b = (Pair(2, 1, 1, 128, 256, "int8", 32, seed=4, meta=True) for _ in range(2))
    x = bf16(np.random.default_rng(1), (2, 200, 2, 128)).cuda()
    ops.kv8_append(a.desc, a.cache, x[:, :, :1], x[:, :, 1:], a.ctx, kmin=a.kmin, kmax=a.kmax)
    for t in range(200):
        ops.kv8_append(b.desc, b.cache, x[:, t:t + 1, :1], x[:, t:t + 1, 1:], b.ctx, kmin=b.kmin, kmax=b.kmax)
    for n in ("k_codes", "v_codes", "k_scales", "v_scales"):
        assert same(getattr(a.cache, n), getattr(b.cache, n)), n
    assert same(a.kmin, b.kmin) and same(a.kmax, b.kmax) and torch.equal(a.ctx, b.ctx)
    assert same(a.cache.k_tail[:, :, :8], b.cache.k_tail[:, :, :8]) and same(a.cache.v_tail[:, :, :8], b.cache.v_tail[:, :, :8])


def test_append_at_capacity_and_clamped_counts():
    p = Pair(3, 1, 1, 64, 64, "e4m3", 16, seed=2)
    p.append([64, 60, 10])
    p.append([1, 4, -3])     # full: unchanged; fills up; negative counts as none
    p.append([0, 1, 99])     # 99 is clamped to the 99 tokens there are, which do not fit
    p.append([1, 1, 54])
    p.check()
    assert p.ctx.tolist() == [64, 64, 64]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_of_zero_infinite_nan_and_tiny_blocks(fmt):
    p = Pair(1, 1, 1, 64, 128, fmt, 16, seed=3)

    def edit(kv):
        kv[0, 0:16] = 0
        kv[0, 20, 0, 3] = float("inf")
        kv[0, 21, 1, 4] = float("nan")
        kv[0, 32:48, 0] *= 2.0 ** -120
        kv[0, 48:64, 1] = kv[0, 48:64, 1] * 0 + 2.0 ** -133  # subnormal
        kv[0, 64:80] *= 2.0 ** 100

    p.append([90], edit)
    p.check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_codes_of_every_magnitude_and_tie(fmt):
    """Every ratio of two 8-bit significands, powers of two and ties among them, in blocks with largest values of all
    significands: each code is that of exact arithmetic."""
    blocks = []
    for a in range(128, 256):
        x = [float(a)] + [s * v * 2.0 ** -k for k in range(10) for v in range(128, 256, 1 + k) for s in (1, -1)]
        x = [v for v in x if abs(v) <= a]
        blocks.append((x + [0.0] * 1024)[:1024])
    x = torch.tensor(blocks, dtype=torch.bfloat16).view(1, 128 * 16, 1, 64)
    assert (x.double().view(128, 1024).abs().max(1).values == torch.arange(128, 256)).all()
    desc = ops.make_desc(1, 1, 1, 64, 16, 128 * 16, torch.bfloat16)
    cache = ops.Kv8Cache.empty(desc, fmt, 16)
    ops.kv8_append(desc, cache, x.cuda(), (-x * 2.0 ** 60).cuda(), ints([0]))
    for codes, scales, ref in ((cache.k_codes, cache.k_scales, x), (cache.v_codes, cache.v_scales, -x * 2.0 ** 60)):
        codes, ref = codes.cpu().numpy().reshape(128, 16, 64), ref.double().numpy().reshape(128, 16, 64)
        for j in range(128):
            want, s = plain.quantise(ref[j], fmt)
            assert (plain.value(codes[j], fmt) == plain.value(want, fmt)).all(), j
            assert float(scales[0, 0, j]) == s


@pytest.mark.parametrize("in_place", [False, True])
def test_append_lengths_in_place_or_apart(in_place):
    p = Pair(3, 1, 1, 64, 256, "int8", 16, seed=9)
    x = bf16(np.random.default_rng(0), (3, 40, 2, 64)).cuda()
    ctx = ints([0, 5, 240])
    out = ctx if in_place else torch.full_like(ctx, -9)
    pos = torch.full_like(ctx, -9)
    got = ops.kv8_append(p.desc, p.cache, x[:, :, :1], x[:, :, 1:], ctx, new_len=ints([40, 0, 17]), ctx_out=out, pos_out=pos)
    assert got is out and out.tolist() == [40, 5, 240] and pos.tolist() == [0, -1, -1]
    none = x[:, :0]
    ops.kv8_append(p.desc, p.cache, none[:, :, :1], none[:, :, 1:], out, pos_out=pos)  # no tokens at all
    assert out.tolist() == [40, 5, 240] and pos.tolist() == [-1, -1, -1]


# ---------------------------------------------------------------- attention

def attention(p, q, pages=None, sink=None, mass_in=None, **kw):
    """Runs the kernel and checks out, lse and the blocks' weight sums row by row."""
    d = p.desc
    mass_out = torch.full_like(p.mass, -5.0) if mass_in is not None else None
    out, lse = ops.kv8_decode_attend(d, p.cache, q.cuda(), p.ctx, page_idx=None if pages is None else pages[0],
                                     count=None if pages is None else pages[1], sink=None if sink is None else sink.cuda(),
                                     mass_in=mass_in, mass_out=mass_out, **kw)
    ops.pipeline_check()
    compare(p, q, out, lse, pages, sink, mass_in, mass_out)
    return out, lse, mass_out


def compare(p, q, out, lse, pages=None, sink=None, mass_in=None, mass_out=None):
    d = p.desc
    G, scale = d.num_q_heads // d.num_kv_heads, d.head_dim ** -0.5
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(d.batch):
        for h in range(d.num_kv_heads):
            row = p.rows[b][h]
            k, v = row.values()
            stored = np.arange(len(row)) < len(row.blocks) * row.block
            if pages is not None:
                r = b * d.num_kv_heads + h
                n = d.capacity if pages[1] is None else int(pages[1][r])
                lst = [int(x) for x in pages[0][r][:max(0, n)] if 0 <= int(x) < d.capacity // d.page_size]
                t = np.concatenate([np.zeros(0, int)] + [np.arange(x * d.page_size, (x + 1) * d.page_size) for x in lst])
                t = t[t < len(row)]
                k, v, stored = k[t], v[t], stored[t]
            heads = slice(h * G, (h + 1) * G)
            qq = q[b, heads].double().numpy()
            ref, ref_lse, w = plain.attend(qq, k, v, scale, None if sink is None else sink[heads].numpy())
            if not np.isfinite(k).all() or not np.isfinite(v).all():
                assert np.isnan(got[b, heads]).any()
                continue
            e, slack = plain.attend_bounds(qq, k, v, scale, w, stored)
            assert (np.abs(got[b, heads] - ref) <= slack + 2.0 ** -8 * (np.abs(ref) + slack) + 1e-37).all(), (
                b, h, np.abs(got[b, heads] - ref).max())
            fin = np.isfinite(ref_lse)
            assert (np.isneginf(got_lse[b, heads]) == ~fin).all()
            assert (np.abs(got_lse[b, heads][fin] - ref_lse[fin]) <= (e + 2.0 ** -20 + 2.0 ** -22 * np.abs(ref_lse))[fin]).all()
            if mass_out is not None:
                n = len(row.blocks)
                m = mass_out[b, h].double().cpu().numpy()
                start = mass_in[b, h, :n].double().cpu().numpy()
                per = w[:, :n * row.block].reshape(G, n, row.block).sum(2)
                tol = 2.0 ** -20 * (start + per.sum(0)) + (per * (2 * e + 2.0 ** -18)[:, None]).sum(0) + 1e-37
                assert (np.abs(m[:n] - start - per.sum(0)) <= tol).all()
                assert (m[n:] == -5).all()


def fill(p, lens):
    while any(int(c) < n for c, n in zip(p.ctx, lens)):
        p.append([min(n - int(c), 200) for c, n in zip(p.ctx, lens)])


def query(p, seed, gain=1.0):
    d = p.desc
    return bf16(np.random.default_rng(seed), (d.batch, d.num_q_heads, d.head_dim), gain)


LENS = [0, 1, 15, 16, 17, 64, 65, 300]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("d,group,hkv,block", [(128, 6, 2, 64), (64, 8, 1, 16), (128, 1, 1, 32), (64, 3, 2, 256), (128, 7, 1, 128)])
@pytest.mark.parametrize("with_sink", [False, True])
def test_attend_dense(fmt, d, group, hkv, block, with_sink):
    p = Pair(len(LENS), group * hkv, hkv, d, 512, fmt, block, seed=d + group)
    fill(p, LENS)
    # values past the context are garbage, NaN codes and NaN tails among it: nothing of it may be seen
    for b, n in enumerate(LENS):
        full = n // block * block
        p.cache.k_codes[b, :, full:] = 0x7f
        p.cache.v_codes[b, :, full:] = 0x7f
        p.cache.k_scales[b, :, full // block:] = float("nan")
        p.cache.v_scales[b, :, full // block:] = float("nan")
        p.cache.k_tail[b, :, n - full:] = float("nan")
        p.cache.v_tail[b, :, n - full:] = float("inf")
    q = query(p, 5, 2.0)
    sink = torch.from_numpy(np.random.default_rng(6).standard_normal(group * hkv)).float() if with_sink else None
    attention(p, q, sink=sink, mass_in=torch.rand_like(p.mass))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("page,block", [(16, 64), (64, 16), (256, 32), (16, 16)])
def test_attend_page_lists(fmt, page, block):
    lens = [0, 5, 200, 511, 512]
    p = Pair(5, 8, 2, 128, 512, fmt, block, page, seed=page)
    fill(p, lens)
    rng = np.random.default_rng(8)
    npg = 512 // page
    idx = np.full((10, npg + 3), -1)
    count = rng.integers(0, npg + 4, 10)
    for r in range(10):
        some = rng.permutation(npg)[:rng.integers(0, npg + 1)]
        idx[r, rng.permutation(npg + 3)[:len(some)]] = some  # any order, gaps anywhere
    count[3] = -4
    attention(p, query(p, 9), pages=(ints(idx), ints(count)))
    attention(p, query(p, 10), pages=(ints(idx), None))


def test_attend_bad_page_ids_are_counted_and_skipped():
    p = Pair(1, 4, 1, 64, 256, "int8", 32, 16, seed=1)
    fill(p, [250])
    idx = ints([[3, 16, -2, 5, 1 << 30, -1, 15]])
    q = query(p, 2)
    out, lse = ops.kv8_decode_attend(p.desc, p.cache, q.cuda(), p.ctx, page_idx=idx)
    with pytest.raises(L.SlsError) as err:
        ops.pipeline_check()
    assert err.value.code == L.SLS_EDEVICE
    compare(p, q, out, lse, (idx, None))
    ops.pipeline_check()


def test_attend_lengths_outside_the_cache_are_clamped():
    p = Pair(2, 4, 1, 64, 128, "e4m3", 32, seed=1)
    fill(p, [128, 0])
    q = query(p, 2)
    ref = ops.kv8_decode_attend(p.desc, p.cache, q.cuda(), p.ctx)[0]
    got = ops.kv8_decode_attend(p.desc, p.cache, q.cuda(), ints([4000, -7]))[0]
    assert torch.equal(got, ref)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_attend_extreme_scales_and_queries(fmt):
    """Blocks whose values differ by a factor of 2^80 next to each other, all-zero blocks, queries of 2^-60 and 2^30."""
    p = Pair(2, 4, 1, 128, 256, fmt, 16, seed=12)

    def edit(kv):
        kv[:, 0:16, 1] *= 2.0 ** -60
        kv[:, 16:32, 1] *= 2.0 ** 20
        kv[:, 32:48] = 0
        kv[:, 48:64, 0] *= 2.0 ** -40
        kv[1, :, 1] *= 2.0 ** -30

    p.append([130, 97], edit)
    q = query(p, 3)
    attention(p, q, mass_in=torch.zeros_like(p.mass))
    q[:, 1] *= 2.0 ** -60
    q[:, 2] *= 2.0 ** 30
    q[:, 3] = 0
    attention(p, q, mass_in=torch.zeros_like(p.mass))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch,cap,lens", [(1, 16, [16]), (1, 16, [5]), (2, 48, [48, 31]), (3, 16, [0, 16, 1])])
def test_attend_caches_smaller_than_a_unit(fmt, d, batch, cap, lens):
    """A whole cache that is smaller than what a warp copies at a time, full to the last slot."""
    p = Pair(batch, 3, 1, d, cap, fmt, 16, page=16, seed=cap + d)
    p.append(lens)
    q = query(p, 8)
    attention(p, q, mass_in=torch.rand_like(p.mass))
    pages = torch.arange(cap // 16, dtype=torch.int32, device="cuda").expand(batch, -1).flip(1).contiguous()
    attention(p, q, pages=(pages, None))


def test_attend_shows_nan_blocks_in_their_row_only():
    p = Pair(2, 4, 2, 64, 128, "int8", 16, seed=3)

    def edit(kv):
        kv[0, 20, 0, 3] = float("inf")  # key of head 0
        kv[1, 5, 3, 3] = float("nan")   # value of head 1

    p.append([60, 60], edit)
    out, lse = ops.kv8_decode_attend(p.desc, p.cache, query(p, 4).cuda(), p.ctx)
    bad = out.isnan().any(-1).cpu()
    assert bad.tolist() == [[True, True, False, False], [False, False, True, True]]
    assert lse[0, :2].isnan().all() and lse[1].isfinite().all()


def test_attend_long_rows_many_rows_and_reused_workspace():
    """Rows of very different length on one workspace, twice (the arrival counters end at zero), with every CTA's
    share crossing rows."""
    lens = [5000, 3, 0, 1200, 17, 2500, 1, 4096]
    p = Pair(8, 8, 2, 64, 5008, "int8", 16, seed=21)
    p.append(lens)
    ws = ops.kv8_attend_workspace(p.desc, p.cache, mass=True)
    a = attention(p, query(p, 1), mass_in=torch.rand_like(p.mass), workspace=ws)
    attention(p, query(p, 2), mass_in=torch.rand_like(p.mass), workspace=ws)
    attention(p, query(p, 3), workspace=ws)  # without sums on the larger workspace
    mass = torch.rand_like(p.mass)
    runs = [ops.kv8_decode_attend(p.desc, p.cache, query(p, 1).cuda(), p.ctx, mass_in=mass, mass_out=torch.zeros_like(mass),
                                  workspace=ws) for _ in range(3)]
    assert all(torch.equal(r[0], a[0]) and torch.equal(r[1], a[1]) for r in runs)  # the same bits every time


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("d,block", [(64, 16), (64, 32), (128, 16), (128, 64)])
@pytest.mark.parametrize("cap", [9216, 262144])  # clusters; ranges
def test_attend_long_uneven_rows(fmt, d, block, cap):
    """Capacities past the cluster kernel's: every CTA takes a range of all rows' tokens, many of them cross rows."""
    lens = [9000, 0, 31, 8001, 1, 257, 4096, 17]
    p = Pair(8, 10, 2, d, cap, fmt, block, seed=d + block)
    p.append(lens)
    ws = ops.kv8_attend_workspace(p.desc, p.cache, mass=True)
    for seed in range(2):
        attention(p, query(p, seed), mass_in=torch.rand_like(p.mass), workspace=ws)
    sink = torch.from_numpy(np.random.default_rng(6).standard_normal(10)).float()
    attention(p, query(p, 7), sink=sink, workspace=ws)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("d,page,block", [(64, 16, 32), (64, 32, 16), (64, 64, 64), (128, 16, 64), (128, 32, 16)])
@pytest.mark.parametrize("batch,hkv", [(2, 2), (45, 2)])  # one cluster per row; more rows than half the GPU's SMs
def test_attend_page_lists_of_few_and_many_rows(fmt, d, page, block, batch, hkv):
    rng = np.random.default_rng(d + page)
    lens = [int(x) for x in rng.integers(0, 321, batch)]
    lens[0] = 320
    p = Pair(batch, 3 * hkv, hkv, d, 320, fmt, block, page, seed=page)
    p.append(lens)
    npg = 320 // page
    idx = np.full((batch * hkv, npg + 2), -1)
    for r in range(batch * hkv):
        some = rng.permutation(npg)[:rng.integers(0, npg + 1)]
        idx[r, rng.permutation(npg + 2)[:len(some)]] = some
    attention(p, query(p, 1), pages=(ints(idx), None))
    attention(p, query(p, 2), pages=(ints(idx), ints(rng.integers(-1, npg + 4, batch * hkv))))
    # in long buffers of lists, of which only the counted entries are read: ranges over all rows
    wide = np.full((batch * hkv, 400000 // page), 1 << 30)
    wide[:, :npg + 2] = idx
    attention(p, query(p, 3), pages=(ints(wide), ints(rng.integers(-1, npg + 3, batch * hkv))))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_attend_more_rows_than_a_cluster_each(fmt):
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 400, 50)]
    p = Pair(50, 16, 2, 64, 400, fmt, 16, seed=8)
    p.append(lens)
    attention(p, query(p, 1), mass_in=torch.rand_like(p.mass))


def test_attend_sums_are_the_same_every_time_and_in_place():
    p = Pair(2, 12, 2, 128, 4096, "e4m3", 64, seed=5)
    p.append([4000, 1111])
    q, m0 = query(p, 6).cuda(), torch.rand_like(p.mass)
    outs = []
    for _ in range(3):
        m = m0.clone()
        ops.kv8_decode_attend(p.desc, p.cache, q, p.ctx, mass_in=m, mass_out=m)
        outs.append(m)
    assert all(same(m, outs[0]) for m in outs)
    none = torch.zeros_like(m0)
    ops.kv8_decode_attend(p.desc, p.cache, q, p.ctx, mass_out=none)  # no earlier sums: from zero
    full = torch.zeros_like(m0)
    ops.kv8_decode_attend(p.desc, p.cache, q, p.ctx, mass_in=torch.zeros_like(m0), mass_out=full)
    assert same(none, full)


def test_attend_past_32_bit_offsets():
    """A cache of 2^25 + 2^20 slots: the last pages' codes lie beyond 2^32 bytes."""
    cap, d = (1 << 25) + (1 << 20), 128
    desc = ops.make_desc(1, 4, 1, d, 64, cap, torch.bfloat16)
    cache = ops.Kv8Cache.empty(desc, "int8", 64)
    rng = np.random.default_rng(2)
    x = bf16(rng, (1, 100, 2, d))
    start = cap - 128
    ctx = ints([start])
    ops.kv8_append(desc, cache, x[:, :, :1].cuda(), x[:, :, 1:].cuda(), ctx)
    assert ctx.tolist() == [start + 100]
    row = plain.PlainCache("int8", 64, d)
    row.append(x[0, :, 0].double().numpy(), x[0, :, 1].double().numpy())
    q = bf16(rng, (1, 4, d))
    idx = ints([[cap // 64 - 2, cap // 64 - 1]])
    out, lse = ops.kv8_decode_attend(desc, cache, q.cuda(), ctx, page_idx=idx)
    k, v = row.values()
    ref, ref_lse, w = plain.attend(q[0].double().numpy(), k, v, d ** -0.5)
    e, slack = plain.attend_bounds(q[0].double().numpy(), k, v, d ** -0.5, w, np.arange(100) < 64)
    assert (np.abs(out[0].double().cpu().numpy() - ref) <= slack + 2.0 ** -8 * (np.abs(ref) + slack)).all()
    assert (np.abs(lse[0].double().cpu().numpy() - ref_lse) <= e + 2.0 ** -19).all()


def test_attend_other_stream_and_two_graphs_with_their_own_workspaces():
    p = Pair(3, 6, 1, 128, 1024, "int8", 64, seed=7)
    p.append([1000, 333, 64])
    q = query(p, 1).cuda()
    ref = ops.kv8_decode_attend(p.desc, p.cache, q, p.ctx)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = ops.kv8_decode_attend(p.desc, p.cache, q, p.ctx)[0]
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, ref)
    graphs = []
    for _ in range(2):
        ws = ops.kv8_attend_workspace(p.desc, p.cache)
        out = torch.zeros_like(ref)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ops.kv8_decode_attend(p.desc, p.cache, q, p.ctx, out=out, workspace=ws, want_lse=False)
        graphs.append((g, out, ws, torch.cuda.Stream()))
    for _ in range(5):
        torch.cuda.synchronize()
        for g, out, _, st in graphs:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for _, out, _, _ in graphs:
            assert torch.equal(out, ref)
            out.zero_()


# ---------------------------------------------------------------- eviction

def choose(mass, n, keep, sinks, recent):
    if n <= keep:
        return list(range(n))
    forced = [j for j in range(n) if j < sinks or j >= n - recent]
    rest = sorted((j for j in range(n) if j not in forced), key=lambda j: (-np.inf if np.isnan(mass[j]) else -mass[j], j))
    nan = [j for j in rest if np.isnan(mass[j])]
    rest = nan + [j for j in rest if not np.isnan(mass[j])]
    return sorted(forced + rest[:keep - len(forced)])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("fmt,d,block,page,meta", [("int8", 128, 64, 16, True), ("e4m3", 64, 16, 16, True),
                                                   ("int8", 64, 32, 32, False), ("e4m3", 128, 16, 4, True)])
@pytest.mark.parametrize("keep,sinks,recent", [(1, 0, 0), (5, 1, 2), (9, 9, 0), (13, 2, 4), (30, 0, 1)])
def test_evict(in_place, fmt, d, block, page, meta, keep, sinks, recent):
    lens = [40 * block + 3, 0, keep * block, (keep + 1) * block + block - 1, 33 * block]
    p = Pair(5, 2, 2, d, 41 * block, fmt, block, page, seed=keep, meta=meta)
    p.append(lens)
    rng = np.random.default_rng(keep)
    mass = rng.random((5, 2, 41)).astype(np.float32)
    mass[:, :, ::3] = 0.25            # ties
    mass[0, 0, 11] = np.nan
    mass[3, 1, 2] = np.inf
    mass[4, 0, 5] = -0.0
    p.mass.copy_(torch.from_numpy(mass))
    old = {n: getattr(p.cache, n).clone() for n in ("k_codes", "v_codes", "k_scales", "v_scales", "k_tail", "v_tail")}
    old_meta = (p.kmin.clone(), p.kmax.clone()) if meta else None
    if in_place:
        ctx = p.ctx.clone()
        _, kept = ops.kv8_evict(p.desc, p.cache, ctx, p.mass, keep, sinks, recent, kmin=p.kmin, kmax=p.kmax)
        to, new_mass, new_meta = p.cache, p.mass, (p.kmin, p.kmax)
    else:
        cap2 = (keep + 2) * block if page <= block else (keep + 2) * block // page * page + page
        desc2 = ops.make_desc(5, 2, 2, d, page, cap2, torch.bfloat16)
        to = ops.Kv8Cache.empty(desc2, fmt, block)
        new_mass = torch.zeros((5, 2, cap2 // block), device="cuda")
        new_meta = tuple(torch.zeros((5, 2, cap2 // page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)) \
            if meta else (None, None)
        ctx, kept = ops.kv8_evict(p.desc, p.cache, p.ctx, p.mass, keep, sinks, recent, dst_desc=desc2, dst=to,
                                  mass_out=new_mass, kmin=p.kmin, kmax=p.kmax, kmin_out=new_meta[0], kmax_out=new_meta[1])
        for n, x in old.items():
            assert same(getattr(p.cache, n), x), n  # the source is only read
    for b, n in enumerate(lens):
        full, rest = n // block, n % block
        assert int(ctx[b]) == min(full, keep) * block + rest
        for h in range(2):
            want = choose(mass[b, h], full, keep, sinks, recent)
            assert kept[b * 2 + h].tolist() == want + [-1] * (keep - len(want))
            for i, j in enumerate(want):
                for nm in ("k_codes", "v_codes"):
                    assert same(getattr(to, nm)[b, h, i * block:(i + 1) * block], old[nm][b, h, j * block:(j + 1) * block])
                for nm in ("k_scales", "v_scales"):
                    assert same(getattr(to, nm)[b, h, i], old[nm][b, h, j])
                assert same(new_mass[b, h, i].cpu(), torch.tensor(mass[b, h, j]))
                if meta:
                    ppb = block // page
                    for x, y in zip(new_meta, old_meta):
                        assert same(x[b, h, i * ppb:(i + 1) * ppb], y[b, h, j * ppb:(j + 1) * ppb])
            for nm in ("k_tail", "v_tail"):
                assert same(getattr(to, nm)[b, h, :rest], old[nm][b, h, :rest])
            if meta:
                ppb, pages = block // page, -(-rest // page)
                for x, y in zip(new_meta, old_meta):
                    assert same(x[b, h, len(want) * ppb:len(want) * ppb + pages], y[b, h, full * ppb:full * ppb + pages])


def test_evict_many_blocks_in_place_equals_out_of_place():
    """Rows of 3000 blocks: several rounds of the moving loop, the lists against a stable sort."""
    p = Pair(2, 1, 1, 64, 48000 + 16, "int8", 16, seed=1)
    x = bf16(np.random.default_rng(0), (2, 48010, 2, 64)).cuda()
    ops.kv8_append(p.desc, p.cache, x[:, :, :1], x[:, :, 1:], p.ctx, new_len=ints([48010, 47000]))
    p.mass.copy_((torch.rand_like(p.mass) * 50).floor())  # many ties
    keep = 1777
    desc2 = ops.make_desc(2, 1, 1, 64, 16, (keep + 1) * 16, torch.bfloat16)
    to = ops.Kv8Cache.empty(desc2, "int8", 16)
    mass2 = torch.zeros((2, 1, keep + 1), device="cuda")
    ctx2, kept2 = ops.kv8_evict(p.desc, p.cache, p.ctx, p.mass, keep, 2, 3, dst_desc=desc2, dst=to, mass_out=mass2)
    for b, n in enumerate([3000, 2937]):
        assert kept2[b].tolist() == choose(p.mass[b, 0].cpu().numpy(), n, keep, 2, 3)
    ctx, kept = ops.kv8_evict(p.desc, p.cache, p.ctx, p.mass, keep, 2, 3)
    assert torch.equal(kept, kept2) and torch.equal(ctx, ctx2)
    for nm, per in (("k_codes", 16), ("v_codes", 16), ("k_scales", 1), ("v_scales", 1)):
        assert same(getattr(p.cache, nm)[:, :, :keep * per], getattr(to, nm)[:, :, :keep * per])
    assert same(p.mass[:, :, :keep], mass2[:, :, :keep])


# ---------------------------------------------------------------- together

def test_prompt_steps_eviction_and_replayed_loop_together():
    """Prompt in two pieces, decode steps with weight sums, an eviction in place, and more steps replayed from a graph,
    against the plain form of every step."""
    B, Hq, H, D, block = 2, 6, 2, 128, 16
    desc = ops.make_desc(B, Hq, H, D, 16, 512, torch.bfloat16)
    rope = ops.make_rope(Hq, H, D, torch.bfloat16, theta=1e5)
    rng = np.random.default_rng(77)
    wq, wk = (1 + 0.1 * bf16(rng, (D,)).float()).to(torch.bfloat16), (1 + 0.1 * bf16(rng, (D,)).float()).to(torch.bfloat16)
    step = ops.Kv8Decode(desc, rope, "int8", block, mass=True, q_weight=wq.cuda(), k_weight=wk.cuda())
    rows = [[plain.PlainCache("int8", block, D) for _ in range(H)] for _ in range(B)]
    seen = [0] * B

    def keys(qkv, n):
        """Appends a piece's rotated keys (the device's own rounding to bf16 is tested elsewhere) to the plain rows."""
        for b in range(B):
            pos = np.arange(seen[b], seen[b] + n[b], dtype=np.int32)
            k = ops.qk_norm_rope(rope, qkv[b, :n[b], :Hq], qkv[b, :n[b], Hq:Hq + H], torch.from_numpy(pos).cuda(),
                                 step.q_weight, step.k_weight)[1].double().cpu().numpy()
            v = qkv[b, :n[b], Hq + H:].double().cpu().numpy()
            for h in range(H):
                rows[b][h].append(k[:, h], v[:, h])
            seen[b] += n[b]

    def check(qkv):
        class P:  # the shape compare() reads
            pass
        p = P()
        p.desc, p.rows, p.ctx = desc, rows, step.ctx_len
        q = step.q.cpu()
        ref, size = plain.norm_rope(qkv[:, :Hq].double().cpu().numpy(), wq.double().numpy(), np.array(seen) - 1, D, False,
                                    [1e5 ** (-2.0 * i / D) for i in range(D // 2)], 1e-6)
        assert (np.abs(q.double().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * size).all()
        compare(p, q, step.out, step.lse)

    for n in ([130, 90], [47, 64]):
        qkv = bf16(rng, (B, max(n), Hq + 2 * H, D)).cuda()
        step.prefill(qkv, ints(n))
        keys(qkv, n)
    loop = harness.Kv8DecodeLoop(step)
    for _ in range(5):
        loop.qkv.copy_(bf16(rng, (B, Hq + 2 * H, D)))
        loop.run_once()
        keys(loop.qkv[:, None], [1, 1])
        check(loop.qkv)
    before, lens = step.mass.clone(), step.ctx_len.tolist()
    kept = step.evict(6, 1, 2).view(B, H, -1).tolist()
    for b in range(B):
        for h in range(H):
            want = choose(before[b, h].cpu().numpy(), lens[b] // block, 6, 1, 2)
            assert kept[b][h] == want
            rows[b][h].blocks = [rows[b][h].blocks[j] for j in want]
    assert step.ctx_len.tolist() == [6 * block + n % block for n in lens] and (step.ctx_len + step.evicted).tolist() == seen
    loop.capture()
    for _ in range(25):  # blocks are completed on the way
        loop.qkv.copy_(bf16(rng, (B, Hq + 2 * H, D)))
        loop.replay()
        keys(loop.qkv[:, None], [1, 1])
        check(loop.qkv)
    ops.pipeline_check()


FIRST_CALLS = """
import torch
from sparse_long_context_gb300 import ops
torch.manual_seed(3)
desc = ops.make_desc(3, 6, 2, 128, 16, 1024, torch.bfloat16)
rope = ops.make_rope(6, 2, 128, torch.bfloat16)
qkv = torch.randn((3, 400, 10, 128), device="cuda").to(torch.bfloat16)
pos = torch.arange(400, dtype=torch.int32, device="cuda")
idx = torch.tensor([[0, 5, 2, -1]] * 6, dtype=torch.int32, device="cuda")

class State:
    def __init__(self):
        self.cache = ops.Kv8Cache.empty(desc, "e4m3", 32)
        self.ctx = torch.zeros(3, dtype=torch.int32, device="cuda")
        self.mass = torch.zeros((3, 2, 32), device="cuda")
        self.ws = ops.kv8_attend_workspace(desc, self.cache, mass=True)

    def run(self):
        q, k = ops.qk_norm_rope(rope, qkv[0, :, :6], qkv[0, :, 6:8], pos)
        ops.kv8_append(desc, self.cache, qkv[:, :, 6:8], qkv[:, :, 8:], self.ctx, mass=self.mass)
        ops.kv8_append(desc, self.cache, qkv[:, :1, 6:8], qkv[:, :1, 8:], self.ctx, mass=self.mass)
        a = ops.kv8_decode_attend(desc, self.cache, qkv[:, 0, :6].contiguous(), self.ctx, mass_in=self.mass,
                                  mass_out=self.mass, workspace=self.ws)
        b = ops.kv8_decode_attend(desc, self.cache, qkv[:, 1, :6].contiguous(), self.ctx, page_idx=idx, workspace=self.ws)
        kept = ops.kv8_evict(desc, self.cache, self.ctx, self.mass, 5, 1, 1)[1]
        return [q, k, *a, *b, kept]

s, g = State(), torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):        # the process's first calls
    out = s.run()
g.replay()
torch.cuda.synchronize()
other = State()
for x, y in zip(out + [s.ctx, s.mass, s.cache.k_codes], other.run() + [other.ctx, other.mass, other.cache.k_codes]):
    assert torch.equal(x, y)
assert s.ctx.tolist() == [5 * 32 + 401 % 32] * 3
ops.pipeline_check()
print("captured")
"""


def test_first_calls_of_a_process_may_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_quest_selection_over_the_8_bit_cache():
    """The sparse step: page min/max kept by the appends, sls_select_pages' lists, attention over them."""
    p = Pair(2, 12, 2, 128, 2048, "e4m3", 64, 16, seed=31, meta=True)
    p.append([1999, 640])
    q = query(p, 8).cuda()
    pages = ops.select_pages(p.desc, q, p.kmin, p.kmax, p.ctx, 24, 1, 64)
    attention(p, q.cpu(), pages=(pages, None))
    rope = ops.make_rope(12, 2, 128, torch.bfloat16)
    step = ops.Kv8Decode(p.desc, rope, "e4m3", 64, k_budget=24, n_sink_pages=1, n_local_tokens=64)
    rng = np.random.default_rng(3)
    step.prefill(bf16(rng, (2, 900, 16, 128)).cuda(), ints([900, 333]))
    for _ in range(3):
        step(bf16(rng, (2, 16, 128)).cuda())
    dense = ops.kv8_decode_attend(p.desc, step.cache, step.q, step.ctx_len)[0]
    listed = ops.kv8_decode_attend(p.desc, step.cache, step.q, step.ctx_len, page_idx=step.page_idx)[0]
    assert torch.equal(listed, step.out) and not torch.equal(dense, listed)
    assert step.ctx_len.tolist() == [903, 336]
