"""fp64 reference of the attention layers' operators (plain numpy and Python lists, row by row; no code shared with the GPU path):
prologue (norm, rotation, cache), its gradients, attention over pages, and the pages' bookkeeping.

    n = w x / sqrt(mean(x^2) + eps),  (y_a, y_b) = (n_a cos - n_b sin, n_b cos + n_a sin),  o = softmax(scale q K^T) V
"""
from __future__ import annotations

import numpy as np

from oracle.ssm import spans  # noqa: F401  (the sequences of a call)


def positions_of(seqs, rows):
    """Index of every row in its sequence (-1: of none)."""
    pos = np.full(rows, -1, dtype=np.int64)
    for lo, hi in seqs:
        pos[lo:hi] = np.arange(hi - lo)
    return pos


def pairs_of(rot, interleaved):
    """(a, b): the elements of each rotated pair."""
    j = np.arange(rot // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)


def rotate(n, pos, freq, interleaved, back=False):
    """n [rows, H, d] turned by its rows' positions."""
    a, b = pairs_of(2 * len(freq), interleaved)
    angle = np.outer(pos.astype(np.float64), freq)[:, None]
    c, s = np.cos(angle), np.sin(angle) * (-1 if back else 1)
    y = n.copy()
    y[..., a], y[..., b] = n[..., a] * c - n[..., b] * s, n[..., b] * c + n[..., a] * s
    return y


def normed(x, w, eps):
    return x if w is None else w * x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def prologue(x, w, freq, pos, eps=1e-6, interleaved=False):
    """One side: x [rows, H, d] -> y."""
    return rotate(normed(x, w, eps), pos, freq, interleaved)


def prologue_grad(x, w, freq, pos, dy, eps=1e-6, interleaved=False):
    """dx and dw (None without w)."""
    dn = rotate(dy, pos, freq, interleaved, back=True)
    if w is None:
        return dn, None
    inv = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh, g = x * inv, dn * w
    return inv * (g - xh * (g * xh).mean(-1, keepdims=True)), (dn * xh).sum((0, 1))


def visible(length, N, n, window):
    """First and last key that token n of a row's newest N sees; none where first > last."""
    last = length - N + n
    return (max(0, last - window + 1) if window else 0), last


def attend(q, k_pages, v_pages, table, lengths, slots, scale, window=0):
    """q [B, N, Hq, d], pools [n_pages, Hkv, page, d] -> o, rows of inactive slots NaN, and the sums of p |v| beside them."""
    B, N, Hq, d = q.shape
    pages, Hkv, page, _ = k_pages.shape
    o, mag = np.full(q.shape, np.nan), np.zeros(q.shape)
    for b in range(B):
        s = b if slots is None else int(slots[b])
        if not 0 <= s < len(table):
            continue
        length = min(max(int(lengths[s]), 0), table.shape[1] * page)
        for n in range(N):
            lo, last = visible(length, N, n, window)
            at = [(int(table[s, t // page]), t % page) for t in range(lo, last + 1)]
            at = [(p, t) for p, t in at if 0 <= p < pages]
            if not at:
                o[b, n] = 0
                continue
            p, t = np.array(at).T
            for h in range(Hq):
                g = h // (Hq // Hkv)
                z = scale * (k_pages[p, g, t] @ q[b, n, h])
                w = np.exp(z - z.max())
                w /= w.sum()
                o[b, n, h], mag[b, n, h] = w @ v_pages[p, g, t], w @ np.abs(v_pages[p, g, t])
    return o, mag


class Pages:
    """The bookkeeping of a cache, request by request."""

    def __init__(self, table, lengths, refs, page):
        self.table, self.lengths, self.refs, self.page = [list(map(int, r)) for r in table], list(map(int, lengths)), list(map(int, refs)), page

    def is_row(self, s):
        return 0 <= s < len(self.table)

    def is_page(self, p):
        return 0 <= p < len(self.refs)

    def length(self, s):
        return min(max(self.lengths[s], 0), len(self.table[s]) * self.page)

    def free(self):
        return [p for p, n in enumerate(self.refs) if n <= 0]

    def release(self, slots):
        for s in filter(self.is_row, slots):
            for p in filter(self.is_page, self.table[s]):
                self.refs[p] -= 1
            self.table[s], self.lengths[s] = [-1] * len(self.table[s]), 0

    def append(self, slots, tokens):
        free, asked, ok, before = self.free(), 0, [], list(self.refs)
        for s, more in zip(slots, tokens):
            good = self.is_row(s) and more >= 0
            have = -(-self.length(s) // self.page) if good else 0
            want = -(-(self.length(s) + more) // self.page) if good else 0
            good = good and want <= len(self.table[s])
            # what the row still names behind its length is its own; where tokens would get to a page that other rows name too, there is no room
            last = self.table[s][have - 1] if good and more > 0 and self.length(s) % self.page else -1
            good = good and not (self.is_page(last) and before[last] > 1)
            while good and have < want and self.is_page(self.table[s][have]) and before[self.table[s][have]] > 0:
                good = before[self.table[s][have]] == 1
                have += good
            first, asked = asked, asked + (want - have if good else 0)
            good = good and (want == have or asked <= len(free))
            if good:
                for i in range(have, want):
                    p = free[first + i - have]
                    self.table[s][i], self.refs[p] = p, 1
                self.lengths[s] = self.length(s) + more
            ok.append(int(good))
        return ok

    def fork(self, src, dst):
        self.release(dst)
        before = [self.length(s) if self.is_row(s) else 0 for s in src]
        free, asked, copies, ok = self.free(), 0, [], []
        for s, t, n in zip(src, dst, before):
            good, copy = self.is_row(s) and self.is_row(t), (-1, -1)
            part = good and n % self.page != 0 and self.is_page(self.table[s][n // self.page])  # a gap stays one
            asked += good and part
            good = good and (not part or asked <= len(free))
            if good and part:
                fresh, last = free[asked - 1], self.table[s][n // self.page]
                self.table[t][n // self.page], self.refs[fresh] = fresh, 1
                copy = (last, fresh)
            copies.append(copy)
            ok.append(int(good))
        for s, t, n, good in zip(src, dst, before, ok):
            if good:
                for i in range(n // self.page):
                    p = self.table[s][i]
                    if self.is_page(p):
                        self.table[t][i] = p
                        self.refs[p] += 1
                self.lengths[t] = n
        return [c[0] for c in copies], [c[1] for c in copies], ok
