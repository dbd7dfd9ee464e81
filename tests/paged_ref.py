"""Plain fp64 forms of the full-attention layers' operators, for the tests: one row, one page and
one table entry at a time."""
import math

import numpy as np
import torch


def half_step(dtype):
    """The largest relative error of one rounding to ``dtype``."""
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ rotary positions
def rope(x, pos, inv_freq, interleaved, scale, inverse=False):
    """(y, |x1| + |x2| per channel) for x [T, H, D] (float64 arrays); angles in extended
    precision (64 bits of mantissa), so that they are good at any int32 position."""
    R = 2 * len(inv_freq)
    a = np.asarray(pos, np.longdouble)[:, None] * np.asarray(inv_freq, np.longdouble)
    two_pi = 2 * np.longdouble("3.14159265358979323846264338327950288")
    a = (a - np.rint(a / two_pi) * two_pi).astype(np.float64)
    c, s = scale * np.cos(a)[:, None], scale * np.sin(a)[:, None] * (-1 if inverse else 1)
    y, size = x.copy(), np.zeros_like(x)
    i1, i2 = (np.arange(0, R, 2), np.arange(1, R, 2)) if interleaved else (np.arange(R // 2), np.arange(R // 2, R))
    x1, x2 = x[..., i1], x[..., i2]
    y[..., i1], y[..., i2] = x1 * c - x2 * s, x2 * c + x1 * s
    size[..., i1] = size[..., i2] = np.abs(x1) + np.abs(x2)
    return y, size


def rope_tol(y, size, scale, dtype):
    """The sine and cosine are fp32: 2^-23 from their own rounding and evaluation, 2^-23 from the
    angle's last rounding (pi 2^-25), 2^-24 from the scale; the two products and their sum 2^-24
    each: together below 2^-21 of scale (|x1| + |x2|). The output is rounded once."""
    return 2.0 ** -21 * abs(scale) * size + half_step(dtype) * np.abs(y) * (1 + 2.0 ** -20) + 1e-38


# ------------------------------------------------------------------ attention
def visible_keys(p, window, pages, page_size, num_pages):
    """Positions that a row at position p sees, in order."""
    lo = max(0, p - window + 1) if window else 0
    hi = min(p, len(pages) * page_size - 1)
    return [j for j in range(lo, hi + 1) if 0 <= pages[j // page_size] < num_pages]


def attention(q, kc, vc, table, lens, cu, scale, window):
    """(o, lse, tol of o, tol of lse), o [T, Hq, D]; rows behind the last sequence are NaN. The tolerances are for inputs
    of kc's type.

    With A = sum_j p_j |v_j| (p the softmax): a score is off by at most ds = scale (D + 2) 2^-24
    sum |q k|; weights, their sum and the products by 2 ds + 2^-20 (the exponential, its argument's rounding at |s| up to 8)
    + 2^-22 |s - max| (the rounding of the exponent's argument) + 2 n 2^-24 (sums over n keys) relative; with bf16 the weights are rounded
    once more (half a step of A); the output is rounded once."""
    dtype = kc.dtype
    T, Hq, D = q.shape
    P, Hk, ps, _ = kc.shape
    G = Hq // Hk
    q, kf, vf = q.double(), kc.double(), vc.double()
    o = torch.full((T, Hq, D), math.nan, dtype=torch.float64)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    for n in range(len(lens)):
        pages = [int(x) for x in table[n]]
        for t in range(cu[n], cu[n + 1]):
            p = int(lens[n]) - (cu[n + 1] - t)
            keys = visible_keys(p, window, pages, ps, P)
            if not keys:
                o[t], lse[t] = 0.0, -math.inf
                continue
            pg = torch.tensor([pages[j // ps] for j in keys])
            at = torch.tensor([j % ps for j in keys])
            k, v = kf[pg, :, at], vf[pg, :, at]  # [keys, Hk, D]
            x = q[t].view(Hk, G, D)
            s = torch.einsum("hgd,khd->hgk", x, k) * scale
            ds = torch.einsum("hgd,khd->hgk", x.abs(), k.abs()).amax(-1) * scale * (D + 2) * 2.0 ** -24
            m = s.amax(-1, keepdim=True)
            w = torch.exp(s - m)
            l = w.sum(-1, keepdim=True)
            w = w / l
            r = torch.einsum("hgk,khd->hgd", w, v)
            A = torch.einsum("hgk,khd->hgd", w, v.abs())
            far = torch.einsum("hgk,khd->hgd", w * (m - s), v.abs())
            rel = (2 * ds + 2.0 ** -20 + 2 * len(keys) * 2.0 ** -24)[..., None]
            half = half_step(dtype)
            tol = rel * A + 2.0 ** -22 * far + half * r.abs() * 1.001 + 1e-37
            if dtype == torch.bfloat16:
                tol = tol + half * A * 1.001
            o[t], to[t] = r.reshape(Hq, D), tol.reshape(Hq, D)
            e = m[..., 0] + torch.log(l[..., 0])
            lse[t] = e.reshape(Hq)
            tl[t] = (ds + 2.0 ** -20 + len(keys) * 2.0 ** -24 + 2.0 ** -22 * e.abs()).reshape(Hq)
    return o, lse, to, tl


# ------------------------------------------------------------------ the cache and its pages
def positions(lens, cu):
    """[(row, sequence, position)] of every new token."""
    return [(t, n, int(lens[n]) - (cu[n + 1] - t)) for n in range(len(lens)) for t in range(cu[n], cu[n + 1])]


class Pages:
    """The bookkeeping with plain lists; ``pools`` are host tensors whose dimension page_dim
    counts the pages."""

    def __init__(self, refs, table, lens, page_size, pools=(), page_dim=0):
        self.refs, self.table, self.lens = list(refs), [list(r) for r in table], list(lens)
        self.ps, self.pools, self.dim = page_size, list(pools), page_dim

    def copy(self, a, b):
        for p in self.pools:
            p.select(self.dim, b).copy_(p.select(self.dim, a))

    def _free(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def _pages(self, n):
        return -(-n // self.ps)

    def _serve(self, needs):
        """needs: pages of each request, None where it is not well formed; the pages that each gets, None if refused."""
        free, at, got = self._free(), 0, []
        for n in needs:
            if n is None:
                got.append(None)
                continue
            got.append(free[at:at + n] if n == 0 or at + n <= len(free) else None)
            at += n
        return got

    def alloc(self, seqs, new):
        N, width, seen, needs = len(self.lens), len(self.table[0]), set(), []
        for s, m in zip(seqs, new):
            ok = 0 <= s < N and s not in seen
            if 0 <= s < N:
                seen.add(s)
            ok = ok and self.lens[s] >= 0 and m >= 0 and self._pages(self.lens[s] + m) <= width
            needs.append(self._pages(self.lens[s] + m) - self._pages(self.lens[s]) if ok else None)
        got = self._serve(needs)
        for s, m, g in zip(seqs, new, got):
            if g is not None:
                have = self._pages(self.lens[s])
                for j, p in enumerate(g):
                    self.table[s][have + j] = p
                    self.refs[p] = 1
                self.lens[s] += m
        return [int(g is not None) for g in got]

    def fork(self, parents, children):
        N, width, seen, needs, was = len(self.lens), len(self.table[0]), set(), [], list(self.lens)
        for a, b in zip(parents, children):
            ok = 0 <= b < N and b not in seen
            if 0 <= b < N:
                seen.add(b)
            ok = ok and 0 <= a < N and was[b] == 0 and was[a] >= 0 and self._pages(was[a]) <= width
            needs.append(int(was[a] % self.ps != 0) if ok else None)
        got = self._serve(needs)
        for a, b, g in zip(parents, children, got):
            if g is None:
                continue
            full = was[a] // self.ps
            for j in range(full):
                p = self.table[b][j] = self.table[a][j]
                if 0 <= p < len(self.refs):
                    self.refs[p] += 1
            if g:
                p = self.table[a][full]
                if 0 <= p < len(self.refs):
                    self.copy(p, g[0])
                self.table[b][full] = g[0]
                self.refs[g[0]] = 1
            self.lens[b] = was[a]
        return [int(g is not None) for g in got]

    def free(self, seqs):
        for s in seqs:
            if 0 <= s < len(self.lens):
                for j in range(min(self._pages(max(0, self.lens[s])), len(self.table[s]))):
                    p = self.table[s][j]
                    if 0 <= p < len(self.refs):
                        self.refs[p] -= 1
                    self.table[s][j] = -1
                self.lens[s] = max(0, self.lens[s]) * 0

    def compact(self):
        to, low, high = {}, 0, len(self.refs) - 1
        while True:
            while low < len(self.refs) and self.refs[low] != 0:
                low += 1
            while high >= 0 and self.refs[high] == 0:
                high -= 1
            if low > high:
                break
            self.refs[low], self.refs[high] = self.refs[high], 0
            self.copy(high, low)
            to[high] = low
        self.table = [[to.get(p, p) for p in r] for r in self.table]
        return len(to)
