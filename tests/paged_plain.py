"""The paged cache in plain form, on the CPU: pages, table and counts as Python and torch values, attention in 64 bits."""
import math

import torch


class PlainPaged:
    def __init__(self, batch, hkv, d, page, cap, k_pages, v_pages, kmin=None, kmax=None):
        self.b, self.h, self.d, self.p, self.cap = batch, hkv, d, page, cap
        self.k, self.v = k_pages.cpu().clone(), v_pages.cpu().clone()
        self.lo, self.hi = (None, None) if kmin is None else (kmin.cpu().clone(), kmax.cpu().clone())
        self.rows = [[] for _ in range(batch)]
        self.ctx = [0] * batch

    @property
    def n(self):
        return self.k.shape[0]

    def refs(self):
        r = [0] * self.n
        for row in self.rows:
            for p in row:
                r[p] += 1
        return r

    def free(self):
        return [p for p, n in enumerate(self.refs()) if n == 0]

    def table(self):
        t = torch.full((self.b, self.cap // self.p), -1, dtype=torch.int32)
        for b, row in enumerate(self.rows):
            t[b, :len(row)] = torch.tensor(row, dtype=torch.int32)
        return t

    def _summary(self, page, n):
        if self.lo is not None:
            self.lo[page], self.hi[page] = self.k[page, :, :n].amin(1), self.k[page, :, :n].amax(1)

    def append(self, k_new, v_new, lens):
        """Returns the first written positions (-1: none)."""
        free, first, pos = self.free(), 0, []
        todo = []
        for b in range(self.b):
            n = min(max(lens[b], 0), k_new.shape[1])
            n = n if self.ctx[b] + n <= self.cap else 0
            need = -(-(self.ctx[b] + n) // self.p) - len(self.rows[b]) if n else 0
            first += need
            ok = n > 0 and (need == 0 or first <= len(free))
            todo.append((n, free[first - need:first]) if ok else (0, []))
            pos.append(self.ctx[b] if ok else -1)
        for b, (n, pages) in enumerate(todo):
            self.rows[b] += pages
            for t in range(n):
                at = self.ctx[b] + t
                page = self.rows[b][at // self.p]
                self.k[page, :, at % self.p], self.v[page, :, at % self.p] = k_new[b, t].cpu(), v_new[b, t].cpu()
            for lp in range(self.ctx[b] // self.p, len(self.rows[b])) if n else ():
                self._summary(self.rows[b][lp], min(self.p, self.ctx[b] + n - lp * self.p))
            self.ctx[b] += n
        return pos

    def fork(self, parent, keep):
        """Returns whether the pages sufficed."""
        lens = []
        for b in range(self.b):
            if not -1 <= parent[b] < self.b:
                lens.append((b, self.ctx[b]))
            else:
                n = self.ctx[parent[b]] if parent[b] >= 0 else 0
                lens.append((parent[b], min(n, max(keep[b], 0)) if keep is not None else n))
        same = [(q == b and n == self.ctx[b]) or (n == 0 and self.ctx[b] == 0) for b, (q, n) in enumerate(lens)]
        whole = {p for b, (q, n) in enumerate(lens)
                 for p in (self.rows[b] if same[b] else self.rows[q][:n // self.p] if n else [])}
        free, rows, copies, kept = self.free(), [], [], set()
        for b, (q, n) in enumerate(lens):
            if same[b]:
                rows.append(list(self.rows[b]))
                continue
            row = self.rows[q][:n // self.p] if n else []
            if n % self.p:
                src = dst = self.rows[q][n // self.p]
                if src in whole or src in kept:
                    if not free:
                        return False
                    dst = free.pop(0)
                kept.add(src)
                copies.append((src, dst, n % self.p))
                row = row + [dst]
            rows.append(row)
        for src, dst, n in copies:
            self.k[dst, :, :n], self.v[dst, :, :n] = self.k[src, :, :n].clone(), self.v[src, :, :n].clone()
            self._summary(dst, n)
        self.rows, self.ctx = rows, [n for _, n in lens]
        return True

    def compact(self):
        """Returns every page's new number (-1: free)."""
        used = [p for p, n in enumerate(self.refs()) if n]
        late, holes = [p for p in used if p >= len(used)], [p for p in self.free() if p < len(used)]
        moved = [-1] * self.n
        for p in used:
            moved[p] = p
        for p, to in zip(late, holes):
            moved[p] = to
            self.k[to], self.v[to] = self.k[p], self.v[p]
            if self.lo is not None:
                self.lo[to], self.hi[to] = self.lo[p], self.hi[p]
        self.rows = [[moved[p] for p in row] for row in self.rows]
        return moved

    def tokens(self, b, j, pages=None):
        """Keys and values [n, D] of sequence b, KV head j: of the context, or of the listed logical pages."""
        n, row = self.ctx[b], self.rows[b]
        if pages is None:
            pages = range(len(row))
        at = [(row[lp], t) for lp in pages if 0 <= lp < len(row) for t in range(min(self.p, n - lp * self.p))]
        p, t = torch.tensor([x for x, _ in at], dtype=torch.long), torch.tensor([x for _, x in at], dtype=torch.long)
        return self.k[p, j, t].double(), self.v[p, j, t].double()

    def attend(self, q, scale, pages=None, sink=None):
        """out [B, Hq, D], lse [B, Hq], and for the tolerances sum of p |v| [B, Hq, D], the largest sum_c |q_c k_c| scale and
        the number of tokens of each head [B, Hq]."""
        hq = q.shape[1]
        g = hq // self.h
        q = q.cpu().double()
        out, size = torch.zeros((self.b, hq, self.d), dtype=torch.float64), torch.zeros((self.b, hq, self.d), dtype=torch.float64)
        lse, dots, count = (torch.zeros((self.b, hq), dtype=torch.float64) for _ in range(3))
        for b in range(self.b):
            for j in range(self.h):
                k, v = self.tokens(b, j, None if pages is None else pages[b * self.h + j])
                for i in range(j * g, (j + 1) * g):
                    x = k @ q[b, i] * scale
                    if sink is not None:
                        x = torch.cat([x, sink[i].cpu().double().view(1)])
                    count[b, i] = k.shape[0]
                    if x.numel() == 0:
                        lse[b, i] = -math.inf
                        continue
                    lse[b, i] = torch.logsumexp(x, 0)
                    p = torch.exp(x[:k.shape[0]] - lse[b, i])
                    out[b, i], size[b, i] = p @ v, p @ v.abs()
                    dots[b, i] = (k.abs() @ q[b, i].abs()).max() * scale if k.shape[0] else 0.0
        return out, lse, size, dots, count


def bounds(dtype, d, out, size, dots, count):
    """How far outputs and lse may be off: the output's rounding (half a step); a score's D products and sums (D + 8 roundings
    of at most dots, 2^-23 each, twice over for the scale and the base-2 exponential's argument), which moves every
    weight by delta relative, and the weights' sum as much; the sums over the tokens (2^-23 each); for bf16 the weights'
    16 bits (2^-15)."""
    delta = (d + 8) * 2.0 ** -22 * dots + 2.0 ** -20
    rel = 2 * delta + count * 2.0 ** -23 + (2.0 ** -15 if dtype == torch.bfloat16 else 0.0)
    return torch.finfo(dtype).eps / 2 * out.abs() + size * rel[..., None] * 1.01 + 1e-30, delta + count * 2.0 ** -23
