"""Bookkeeping of pages that rows share and one of them is shortened into, in the reference (CPU only): no row writes a shared page."""
import numpy as np

from oracle import attn
from tests.test_pages_shortened_oracle import in_order


def test_the_last_page_is_shared():
    """Shortened into a page that its fork names: no room for tokens there, but for a copy of the row."""
    p = attn.Pages(np.full((3, 4), -1), np.zeros(3), np.zeros(9), 4)
    p.append([0], [12])
    p.fork([0], [1])
    p.lengths[0] = 10
    before = [list(r) for r in p.table], list(p.lengths), list(p.refs)
    assert p.append([0, 1], [1, 0]) == [0, 1] and (p.table, p.lengths, p.refs) == before
    assert p.append([0], [0]) == [1]
    _, to, ok = p.fork([0], [2])
    assert ok == [1] and to == [p.table[2][2]] and to[0] not in p.table[1]
    p.release([0])
    assert p.append([2, 1], [5, 1]) == [1, 1]
    in_order(p)


def test_tokens_go_to_pages_of_one_row():
    """Whatever is appended, forked, shortened and given back: the pages that an append's tokens lie in have one row."""
    rng = np.random.default_rng(6)
    p = attn.Pages(np.full((6, 5), -1), np.zeros(6), np.zeros(20), 4)
    turned_down = 0
    for _ in range(600):
        kind, a = rng.integers(4), rng.permutation(6)
        if kind == 0:
            more, had = rng.integers(0, 7, 3), [p.lengths[s] for s in a[:3]]
            for s, n, m, ok in zip(a, had, more, p.append(a[:3], more)):
                assert p.lengths[s] == n + ok * m
                turned_down += not ok
                if ok and m:
                    assert all(p.refs[p.table[s][i]] == 1 for i in range(n // 4, -(-(n + m) // 4)))
        elif kind == 1:
            p.fork(a[:2], a[2:4])
        elif kind == 2:
            p.lengths[a[0]] = int(rng.integers(0, p.lengths[a[0]] + 1))
        else:
            p.release(a[:1])
        in_order(p)
    assert 20 < turned_down < 400
