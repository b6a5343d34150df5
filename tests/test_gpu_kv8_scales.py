"""Precision of the 8-bit attend's value product: values of any size next to a tail, weights far below the largest, and
tail weights, against the plain 64-bit form with bounds that do not depend on the values' size."""
import numpy as np
import pytest
import torch

from sparse_long_context_gb300 import ops
from tests import kv8_plain as plain
from tests.test_gpu_kv8 import Pair, bf16, ints, query

pytestmark = pytest.mark.gpu


def value_sizes(row, block, fmt):
    """Per token the largest magnitude that its value scale stands for: of its block, or of its group of 16 in the tail."""
    out = [np.repeat(float(vs) * plain.TOP[fmt], block) for _, _, _, vs in row.blocks]
    for g in range(0, len(row.tail_v), 16):
        x = np.abs(np.array(row.tail_v[g:g + 16]))
        out.append(np.full(len(x), x.max()))
    return np.concatenate([np.zeros(0)] + out)


def bounds(q, k, v, scale, p, stored, size):
    """Bounds of the kernel's errors from its formula's roundings, relative to the values' own size.
    Scores: as in plain.attend_bounds.  A stored token's weight is rounded to fp16: half a step is 2^-11 of it, or, among
    the subnormals, 2^-25 in units in which the token with the largest product of weight and value scale has
    2^14 or more, so 2^-39 of the largest weight times value for each token.  A tail token's weight is the sum of a
    truncated bf16 (the rest is below 2^-7 of it) and that rest in bf16 (half a step is 2^-8 of it): 2^-15.
    Sums: a warp adds its tokens' groups one after the other (a row is spread over 12 warps at least), then up to 200
    partials are merged, each addition off by 2^-23 of at most sum p |v| (truncating adds), in the accumulators and
    in the weights' sum alike."""
    d, n = q.shape[1], k.shape[0]
    e = d * 2.0 ** -23 * scale * (np.abs(q) @ np.abs(k).T).max(1)
    pv = p @ np.abs(v)
    w = (p * np.where(stored, 2.0 ** -11, 2.0 ** -15)) @ np.abs(v)
    adds = 2 * (n / 192 + 200) * 2.0 ** -23
    return e, w + (2 * e[:, None] + 2.0 ** -20 + adds) * pv + n * 2.0 ** -39 * (p * size).max(1)[:, None]


def check(p, q, pages=None, **kw):
    d = p.desc
    G, scale = d.num_q_heads // d.num_kv_heads, d.head_dim ** -0.5
    out, lse = ops.kv8_decode_attend(d, p.cache, q.cuda(), p.ctx, page_idx=None if pages is None else pages[0],
                                     count=None if pages is None else pages[1], **kw)
    ops.pipeline_check()
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(d.batch):
        for h in range(d.num_kv_heads):
            row = p.rows[b][h]
            if not len(row):
                continue
            k, v = row.values()
            size = value_sizes(row, row.block, row.fmt)
            stored = np.arange(len(row)) < len(row.blocks) * row.block
            if pages is not None:
                r = b * d.num_kv_heads + h
                n = pages[0].shape[1] if pages[1] is None else int(pages[1][r])
                lst = [int(x) for x in pages[0][r][:n] if int(x) >= 0]
                t = np.concatenate([np.zeros(0, int)] + [np.arange(x * d.page_size, (x + 1) * d.page_size) for x in lst])
                t = t[t < len(row)]
                k, v, stored, size = k[t], v[t], stored[t], size[t]
            at = slice(h * G, (h + 1) * G)
            qq = q[b, at].double().numpy()
            ref, ref_lse, w = plain.attend(qq, k, v, scale)
            e, slack = bounds(qq, k, v, scale, w, stored, size)
            err = np.abs(got[b, at] - ref)
            assert (err <= slack + 2.0 ** -8 * (np.abs(ref) + slack)).all(), (b, h, (err / (np.abs(ref) + slack)).max())
            assert (np.abs(got_lse[b, at] - ref_lse) <= e + 2.0 ** -18 + 2.0 ** -22 * np.abs(ref_lse)).all()


SCALES = [-14, -20, -30, 30]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", SCALES)
def test_small_values_after_a_tail_one_cta_per_row(fmt, d, power):
    """128 rows in a capacity of 4096: a row is one CTA's, whose last warps start with the tail."""
    p = Pair(128, 2, 1, d, 4096, fmt, 64, seed=d)
    p.append([3000 + 37 * b if b < 4 else b % 3 for b in range(128)], lambda kv: kv[:, :, 1].mul_(2.0 ** power))
    check(p, query(p, 1))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", SCALES)
def test_small_values_after_a_tail_in_ranges(fmt, d, power):
    """Two rows of 90000 tokens in a deep cache: ranges of 18 or 37 units a CTA, for 12 warps."""
    p = Pair(1, 6, 2, d, 262144, fmt, 256, seed=d + 1)
    p.append([90001 + 254], lambda kv: kv[:, :, 2:].mul_(2.0 ** power))
    check(p, query(p, 2))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("power", SCALES)
def test_small_values_after_a_listed_tail(fmt, d, page, power):
    """The page with the tail comes first in the list, so the warp that holds it goes on to stored units (a cluster of 16
    CTAs has 20 to 40 units each for its 12 warps)."""
    cap = 20032
    npg = cap // page
    p = Pair(1, 4, 1, d, cap, fmt, 64, page, seed=d + 2)
    p.append([cap - 23], lambda kv: kv[:, :, 1].mul_(2.0 ** power))
    order = [npg - 1] + list(np.random.default_rng(3).permutation(npg - 1))
    check(p, query(p, 3), pages=(ints([order]), None))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("power", [-24, 0])
def test_tail_and_blocks_of_different_sizes(fmt, power):
    """A tail whose values are far larger, or far smaller, than the blocks' (both outweigh the other by logits)."""
    p = Pair(128, 2, 1, 128, 4096, fmt, 64, seed=9)

    def edit(kv):
        kv[0, :2944, 1] *= 2.0 ** (power - 10)
        kv[1, :2944, 1] *= 2.0 ** power
        kv[1, 2944:, 1] *= 2.0 ** (power - 20)
        kv[2, 2944:, 1] = 0       # an all-zero tail
        kv[3, :2944, 1] = 0       # all-zero blocks

    p.append([3000 if b < 4 else 1 for b in range(128)], edit)
    check(p, query(p, 4))


def test_infinite_tail_value_shows_in_its_channel_only():
    p = Pair(128, 2, 1, 128, 4096, "int8", 64, seed=10)

    def edit(kv):
        kv[0, 2990, 1, 5] = float("inf")
        kv[1, 2991, 1, 6] = float("-inf")
        kv[2, 2992, 1, 7] = float("nan")

    p.append([3000 if b < 4 else 1 for b in range(128)], edit)
    q = query(p, 5)
    out = ops.kv8_decode_attend(p.desc, p.cache, q.cuda(), p.ctx)[0].cpu()
    assert (out[0, :, 5] == float("inf")).all() and (out[1, :, 6] == float("-inf")).all() and out[2, :, 7].isnan().all()
    for b, ch in ((0, 5), (1, 6), (2, 7)):  # the other channels: as with a zero there
        row = p.rows[b][0]
        k, v = row.values()
        v = v.copy()
        v[~np.isfinite(v)] = 0
        qq = q[b].double().numpy()
        ref, _, w = plain.attend(qq, k, v, 128 ** -0.5)
        stored = np.arange(len(row)) < 2944
        row.tail_v = [np.where(np.isfinite(x), x, 0) for x in row.tail_v]
        _, slack = bounds(qq, k, v, 128 ** -0.5, w, stored, value_sizes(row, 64, "int8"))
        err = np.abs(out[b].double().numpy() - ref)
        err[:, ch] = 0
        assert (err <= slack + 2.0 ** -8 * (np.abs(ref) + slack)).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gap,at", [(14, 5), (18, 5), (18, 6800), (22, 5)])
def test_weights_far_below_a_dominant_token(fmt, d, gap, at):
    """One token without a value of its own draws nearly all of the weight; the others have about e^-gap of it each, and all
    of the output is theirs.  128 rows in a capacity of 6912, one CTA each: the dominant token's warp has a twelfth of
    its row, whose weights are relative to it."""
    lens = [6900, 6912, 6801] + [1] * 125
    p = Pair(128, 2, 1, d, 6912, fmt, 64, seed=gap)
    q = torch.zeros((128, 2, d), dtype=torch.bfloat16)
    q[:, :, 0] = d ** 0.5  # the logit is the key's first channel, nearly (8 and 11.3125)

    def edit(kv):
        kv[:3, :, 0, 0] = torch.from_numpy(np.random.default_rng(1).standard_normal((3, 6912)) * 0.5).to(torch.bfloat16)
        kv[:3, at, 0, 0] = gap
        kv[:3, :, 1] = kv[:3, :, 1].abs()
        kv[:3, at, 1] = 0

    p.append(lens, edit)
    check(p, q)


@pytest.mark.parametrize("d", [64, 128])
def test_tail_weights_near_cancellation(d):
    """Rows that are nothing but tail, with values +1 and -1: the output is the difference of sums of weights."""
    lens = [1, 2, 3, 15, 16, 17, 100, 255]
    p = Pair(len(lens), 8, 1, d, 512, "int8", 256, seed=d + 5)

    def edit(kv):
        kv[:, 0::2, 1] = 1
        kv[:, 1::2, 1] = -1
        kv[:, 1::2, 0] = kv[:, 0::2, 0][:, :kv[:, 1::2].shape[1]] * 1.0078125  # logits in pairs almost alike

    p.append(lens, edit)
    check(p, query(p, 6, 0.25))
