"""Bookkeeping of pages where rows are shortened, in the reference (CPU only): no page is lost, none is written by two rows."""
import numpy as np
import pytest

from oracle import attn


def in_order(p):
    """Every count is the number of entries that name its page, and rows hold the pages of their tokens."""
    entries = [e for row in p.table for e in row if e >= 0]
    assert p.refs == [entries.count(i) for i in range(len(p.refs))]
    for row, n in zip(p.table, p.lengths):
        assert all(e >= 0 for e in row[:-(-n // p.page)])


@pytest.mark.parametrize("page", [1, 4, 16])
def test_drafts_turned_down(page):
    """Four tokens drafted, none to four of them taken back, over many pages' ends: as many pages as the longest row took."""
    rng = np.random.default_rng(page)
    p = attn.Pages(np.full((2, 60), -1), np.zeros(2), np.zeros(100), page)
    most = 0
    for _ in range(40):
        if p.lengths[0] + 4 > 60 * page:
            break
        assert p.append([0], [4]) == [1]
        most = max(most, p.lengths[0])
        p.lengths[0] -= int(rng.integers(0, 5))
        in_order(p)
        assert sum(p.refs) == -(-most // page)
    p.release([0, 1])
    assert not any(p.refs)


def test_the_last_free_page():
    """A full cache: a row that gave tokens back has its own page to go on with."""
    p = attn.Pages(np.full((2, 3), -1), np.zeros(2), np.zeros(3), 4)
    assert p.append([0, 1], [5, 4]) == [1, 1]
    p.lengths[0] = 3
    assert p.append([0], [2]) == [1] and p.append([1], [1]) == [0] and p.append([0], [4]) == [0]
    in_order(p)


def test_pages_that_others_name():
    """A row shortened to before its fork does not write into what it shares; a fork of it does not hold those pages."""
    p = attn.Pages(np.full((3, 4), -1), np.zeros(3), np.zeros(9), 4)
    p.append([0], [12])
    p.fork([0], [1])
    p.lengths[0] = 4
    before = [list(r) for r in p.table], list(p.lengths), list(p.refs)
    assert p.append([0], [1]) == [0] and (p.table, p.lengths, p.refs) == before
    assert p.append([0], [0]) == [1]
    p.fork([0], [2])
    p.release([0])
    assert p.append([2], [6]) == [1]
    in_order(p)
    assert not set(p.table[2][1:3]) & set(p.table[1])
