"""The pages of a cache on the GPU against their bookkeeping request by request (oracle/attn.Pages): whole numbers, equal to the last one."""
import numpy as np
import pytest

from oracle import attn
from tests.test_gpu_attn_prologue import _int32, g2  # noqa: F401

pytestmark = pytest.mark.gpu


class Both:
    """A cache on the device and its reference."""

    def __init__(self, g2, rows, wide, pages, page):  # noqa: F811
        self.g2, self.page = g2, page
        self.ref = attn.Pages(np.full((rows, wide), -1), np.zeros(rows, int), np.zeros(pages, int), page)
        self.put()

    def put(self):
        self.dev = (_int32(self.ref.table), _int32(self.ref.lengths), _int32(self.ref.refs))

    def same(self, *pairs):
        for got, want in zip(self.dev, (self.ref.table, self.ref.lengths, self.ref.refs)):
            np.testing.assert_array_equal(got.cpu().numpy(), np.array(want))
        for got, want in pairs:
            np.testing.assert_array_equal(got.cpu().numpy(), np.array(want))

    def append(self, slots, tokens):
        n = len(slots)
        got = self.g2.pages_append(*self.dev, _int32(slots), tokens if isinstance(tokens, int) else _int32(tokens), page=self.page)
        self.same((got, self.ref.append(list(map(int, slots)), [tokens] * n if isinstance(tokens, int) else list(map(int, tokens)))))

    def fork(self, src, dst):
        got = self.g2.pages_fork(*self.dev, _int32(src), _int32(dst), page=self.page)
        self.same(*zip(got, self.ref.fork(list(map(int, src)), list(map(int, dst)))))

    def release(self, slots):
        self.g2.pages_release(*self.dev, _int32(slots))
        self.ref.release(list(dict.fromkeys(map(int, slots))))
        self.same()


@pytest.mark.parametrize("rows,wide,pages,page", [(1, 1, 1, 1), (4, 3, 7, 16), (40, 9, 200, 24), (300, 20, 3000, 8), (30, 700, 70000, 4)])
def test_requests_in_any_order(g2, rows, wide, pages, page):  # noqa: F811
    rng = np.random.default_rng(rows)
    b = Both(g2, rows, wide, pages, page)
    for i in range(25):
        order = rng.permutation(rows)
        n, m = rng.integers(1, rows + 1), rng.integers(0, rows // 2 + 1)
        b.append(order[:n], rng.integers(0, 2 * page + 2, n))
        if m:
            b.fork(rng.choice(order[m:], m), order[:m])
        b.append(order[:n], int(rng.integers(0, 3)))
        if i % 3 == 2:
            b.release(order[:rng.integers(1, rows + 1)])


def test_more_requests_than_threads(g2):  # noqa: F811
    """2500 requests against pages that run out in their midst."""
    rng = np.random.default_rng(1)
    b = Both(g2, 5000, 4, 3000, 8)
    b.append(rng.permutation(5000)[:2500], rng.integers(0, 25, 2500))
    b.append(np.arange(5000), 1)
    b.release(np.arange(0, 5000, 3))
    b.fork(np.arange(1, 5000, 6)[:833], np.arange(3, 5000, 6))


def test_requests_that_cannot_be_met(g2):  # noqa: F811
    b = Both(g2, 6, 3, 5, 4)
    b.append([0, 9, 1, -1, 2], [4, 4, -1, 4, 100])     # no such row, fewer than no tokens, more than the table names
    b.append([1, 2, 3], [9, 4, 0])                     # three of four pages left; then one; none asked for
    b.append([4, 3], [4, 2])                           # none left
    b.release([1, 1, 77, -4])                          # listed twice: given back once
    b.append([4], [2])
    b.fork([4, 0, 8, 0], [5, 3, 1, 60])                # sources and rows that are none
    b.fork([4, 5, 2], [0, 1, 3])
    b.fork([0, 4], [4, 0])                             # a source that is emptied first counts as empty
    b.append([], [])
    b.fork([], [])
    b.release([])
    b.append([0], 2 ** 31 - 1)


def test_values_out_of_range(g2):  # noqa: F811
    """Tables, lengths and counts that no call leaves: clamped or passed over."""
    rng = np.random.default_rng(2)
    b = Both(g2, 8, 4, 20, 4)
    b.ref.table = rng.integers(-3, 30, (8, 4)).tolist()
    b.ref.lengths = [-7, 2 ** 31 - 1, 5, 16, 17, 0, 3, -2 ** 31]
    b.ref.refs = rng.integers(-2, 3, 20).tolist()
    b.put()
    b.fork([1, 2, 3], [0, 6, 5])
    b.append([7, 2, 3, 4], [3, 1, 1, 1])
    b.release([1, 2])


@pytest.mark.parametrize("width", [1, 3, 8, 100, 4096, 8192 * 2 + 4, 100_001])
@pytest.mark.parametrize("dtype", ["uint8", "bfloat16", "float32"])
def test_copies(g2, width, dtype):  # noqa: F811
    import torch

    rng = np.random.default_rng(width)
    pools = [torch.randint(0, 250, (37, width * m), device="cuda").to(getattr(torch, dtype)) for m in (1, 2)]
    order = rng.permutation(37)
    src, dst = order[:12].copy(), order[20:32].copy()
    src[3], dst[5], src[7], dst[8] = -1, -1, 37, 2 ** 31 - 1
    want = [p.clone() for p in pools]
    good = [(a, b) for a, b in zip(src, dst) if 0 <= a < 37 and 0 <= b < 37]
    for p in want:
        p[[b for _, b in good]] = p[[a for a, _ in good]]
    g2.pages_copy(pools, _int32(src), _int32(dst))
    assert all(torch.equal(a, b) for a, b in zip(pools, want))


def test_many_pools_and_none(g2):  # noqa: F811
    import torch

    pools = [torch.randn(5, 3 + i, device="cuda") for i in range(71)]
    want = [p.clone() for p in pools]
    for p in want:
        p[4] = p[1]
    g2.pages_copy(pools, _int32([1]), _int32([4]))
    assert all(torch.equal(a, b) for a, b in zip(pools, want))
    g2.pages_copy([], _int32([1]), _int32([4]))
    g2.pages_copy(pools, _int32([]), _int32([]))
    g2.pages_copy([torch.empty(0, 4, device="cuda")], _int32([1]), _int32([4]))
    assert all(torch.equal(a, b) for a, b in zip(pools, want))


def test_copies_of_long_rows(g2):  # noqa: F811
    """Rows behind 2^32 bytes, in several pieces each."""
    import torch

    pool = torch.empty(3, 700_000_001, dtype=torch.float32, device="cuda")
    pool[0].fill_(1)
    pool[2].fill_(5)
    pool[2, -1] = 9
    g2.pages_copy([pool], _int32([2]), _int32([1]))
    assert torch.equal(pool[1], pool[2]) and bool((pool[0] == 1).all())


def test_captured(g2):  # noqa: F811
    """A step's calls in a graph: each replay goes on from what the last one left."""
    import torch

    b = Both(g2, 6, 8, 40, 4)
    b.append([0, 1, 2], [5, 9, 13])
    pool = torch.arange(40, device="cuda", dtype=torch.float32)[:, None].repeat(1, 8)
    src, dst, rows = _int32([0, 1]), _int32([3, 4]), _int32([3, 4, 2])

    def step():
        a, c, ok = g2.pages_fork(*b.dev, src, dst, page=4)
        g2.pages_copy([pool], a, c)
        return a, c, ok, g2.pages_append(*b.dev, rows, 1, page=4)

    kept = [t.clone() for t in b.dev]
    step()
    for t, k in zip(b.dev, kept):
        t.copy_(k)
    pool.copy_(torch.arange(40, device="cuda")[:, None].repeat(1, 8))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    want = pool.clone()
    for _ in range(5):
        graph.replay()
        copies = b.ref.fork([0, 1], [3, 4])
        ok = b.ref.append([3, 4, 2], [1, 1, 1])
        for x, y in zip(*copies[:2]):
            if y >= 0:
                want[y] = want[x]
        b.same(*zip(got, (*copies, ok)))
        assert torch.equal(pool, want)
