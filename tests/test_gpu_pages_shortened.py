"""Rows that are shortened and go on, on the GPU against their bookkeeping request by request: whole numbers, equal to the last one."""
import numpy as np
import pytest

from tests.test_gpu_attn_prologue import _int32, g2  # noqa: F401
from tests.test_gpu_pages import Both
from tests.test_pages_shortened_oracle import in_order

pytestmark = pytest.mark.gpu


def shorten(b, row, length):
    b.ref.lengths[row] = length
    b.dev[1][row] = length


@pytest.mark.parametrize("rows,wide,pages,page", [(2, 30, 50, 4), (40, 9, 200, 24), (300, 20, 3000, 8), (12, 700, 5000, 4)])
def test_any_order(g2, rows, wide, pages, page):  # noqa: F811
    """Requests, forks, rows shortened by a token, by pages and to nothing, to before their forks too, and pages that run out."""
    rng = np.random.default_rng(rows)
    b = Both(g2, rows, wide, pages, page)
    for i in range(30):
        order = rng.permutation(rows)
        n, m = rng.integers(1, rows + 1), rng.integers(0, rows // 3 + 1)
        b.append(order[:n], rng.integers(0, (wide if i % 5 == 0 else 3) * page + 2, n))
        if m:
            b.fork(rng.choice(order[m:], m), order[:m])
        for row in order[:n]:
            shorten(b, row, max(0, b.ref.lengths[row] - int(rng.choice([0, 1, 3, page, 2 * page + 1, 10 ** 6], p=[.3, .3, .2, .1, .05, .05]))))
        b.append(order[::2], int(rng.integers(0, page + 2)))
        in_order(b.ref)
        if i % 4 == 3:
            b.release(order[:rng.integers(1, rows + 1)])
    b.release(np.arange(rows))
    assert not any(b.ref.refs)


def test_drafts_in_a_graph(g2):  # noqa: F811
    """Four tokens drafted for each row and some taken back, on the device, captured once and replayed over many pages' ends."""
    import torch

    b = Both(g2, 3, 40, 70, 4)
    b.append([0, 1, 2], [3, 4, 6])
    slots, back = _int32([2, 0, 1]), _int32([0, 0, 0])

    def step():
        ok = g2.pages_append(*b.dev, slots, 4, page=4)
        b.dev[1].index_add_(0, slots, -back)
        return ok

    kept = [t.clone() for t in b.dev]
    step()
    for t, k in zip(b.dev, kept):
        t.copy_(k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ok = step()
    rng = np.random.default_rng(3)
    for _ in range(30):
        turned_down = rng.integers(0, 5, 3)
        back.copy_(_int32(turned_down))
        graph.replay()
        want = b.ref.append([2, 0, 1], [4, 4, 4])
        for s, n in zip([2, 0, 1], turned_down):
            b.ref.lengths[s] -= int(n)
        b.same((ok, want))
        in_order(b.ref)
    b.release([0, 1, 2])
    assert not any(b.ref.refs)
