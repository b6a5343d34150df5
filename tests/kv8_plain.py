"""Plain 64-bit implementations of the 8-bit cache's operators (numpy, loops in the order of the definitions), the
reference of tests/test_gpu_kv8.py and tests/test_gpu_qk_rope.py."""
import math

import numpy as np

TOP = {"int8": 127.0, "e4m3": 448.0}


def e4m3_table():
    """Values of the codes 0..126 (4-bit exponent with bias 7, 3-bit mantissa, subnormals below 2^-6)."""
    out = []
    for c in range(127):
        e, m = c >> 3, c & 7
        out.append(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(out)


E4M3 = e4m3_table()


def e4m3_code(y):
    """Nearest code of float64 values with |y| <= 448, ties to the even code."""
    mag = np.abs(y)
    hi = np.clip(np.searchsorted(E4M3, mag), 0, 126)   # first code with value >= mag
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = mag - E4M3[lo], E4M3[hi] - mag
    code = np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)
    return (code | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def value(codes, fmt):
    if fmt == "int8":
        return codes.view(np.int8).astype(np.float64)
    return np.where(codes & 128, -1.0, 1.0) * E4M3[np.minimum(codes & 127, 126)]


def quantise(x, fmt):
    """Codes and scale of one block [block, D] of float64 values that are bf16 numbers."""
    if not np.isfinite(x).all():
        return np.zeros(x.shape, np.uint8), np.float32(np.nan)
    amax = np.abs(x).max()
    if amax == 0:
        return np.zeros(x.shape, np.uint8), np.float32(0)
    y = x * TOP[fmt] / amax  # exact product, one rounding; a tie of the exact quotient stays one
    codes = np.rint(y).astype(np.int8).view(np.uint8) if fmt == "int8" else e4m3_code(y)
    return codes, np.float32(np.float32(amax) / np.float32(TOP[fmt]))


class PlainCache:
    """One (sequence, KV head) row: every token ever appended and not evicted, as the cache should hold it."""

    def __init__(self, fmt, block, d):
        self.fmt, self.block, self.d = fmt, block, d
        self.blocks = []                      # (k codes, k scale, v codes, v scale)
        self.tail_k, self.tail_v = [], []

    def __len__(self):
        return len(self.blocks) * self.block + len(self.tail_k)

    def append(self, k, v):
        for a, b in zip(k, v):
            self.tail_k.append(a)
            self.tail_v.append(b)
            if len(self.tail_k) == self.block:
                kc, ks = quantise(np.array(self.tail_k), self.fmt)
                vc, vs = quantise(np.array(self.tail_v), self.fmt)
                self.blocks.append((kc, ks, vc, vs))
                self.tail_k, self.tail_v = [], []

    def values(self):
        ks = [value(kc, self.fmt) * float(s) for kc, s, _, _ in self.blocks]
        vs = [value(vc, self.fmt) * float(s) for _, _, vc, s in self.blocks]
        empty = [np.zeros((0, self.d))]
        return (np.concatenate(empty + ks + ([np.array(self.tail_k)] if self.tail_k else [])),
                np.concatenate(empty + vs + ([np.array(self.tail_v)] if self.tail_v else [])))


def norm_rope(x, w, pos, rot, inter, freq, eps):
    """x [N, H, D] float64; returns the result and, per element, |y_a| + |y_b| of its pair (the size that the
    rotation's rounding errors are relative to)."""
    y = np.array(x, np.float64)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * w
    out, size = y.copy(), np.abs(y)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        # the angle modulo one turn in exact integer arithmetic on the frequency's own bits
        num, den = float(freq[i] / (2 * math.pi)).as_integer_ratio()
        turn = np.array([((int(p) * num) % den) / den for p in pos])
        c, s = np.cos(2 * math.pi * turn)[:, None], np.sin(2 * math.pi * turn)[:, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
        size[..., a] = size[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    return out, size


def attend(q, k, v, scale, sink=None):
    """q [G, D] over k, v [n, D]: out [G, D], lse [G], weights [G, n] (the sink in the normaliser)."""
    x = q @ k.T * scale
    full = x if sink is None else np.concatenate([x, np.asarray(sink, np.float64)[:, None]], 1)
    if full.shape[1] == 0:
        return np.zeros((q.shape[0], v.shape[1])), np.full(q.shape[0], -np.inf), x
    m = full.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        total = np.exp(full - m).sum(1, keepdims=True)
        p = np.exp(x - m) / total
        return p @ v, (m + np.log(total))[:, 0], p


def attend_bounds(q, k, v, scale, p, stored):
    """Bounds of the kernel's errors, from its formula's roundings.  Scores: a sum of D fp32 products is off by at most
    D 2^-23 sum |q k| (with truncating adds).  A score error e changes a weight by the factor exp(2 e).  Weights
    enter the value product rounded to fp16 (half a step, 2^-11; in the tail to bf16, 2^-8), and weights far
    below the largest in fp16's subnormals (2^-24 of the largest value at most).  The output is rounded to bf16."""
    d, n = q.shape[1], k.shape[0]
    e = (d * 2.0 ** -23 * scale * (np.abs(q) @ np.abs(k).T).max(1)) if n else np.zeros(q.shape[0])
    pv = p @ np.abs(v)
    w = (p * np.where(stored, 2.0 ** -11, 2.0 ** -8)) @ np.abs(v)
    vmax = np.abs(v).max() if n else 0.0
    slack = w + (2 * e[:, None] + 2.0 ** -20) * pv + n * 2.0 ** -24 * vmax
    return e, slack
