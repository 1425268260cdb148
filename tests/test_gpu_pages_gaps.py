"""Forks of rows whose tables name no page in some places, the last one among them: the fork answers as its source does."""
import numpy as np
import pytest

from tests.test_gpu_attn_prologue import _dev, _int32, g2  # noqa: F401
from tests.test_gpu_pages import Both

pytestmark = pytest.mark.gpu


def test_a_gap_stays_one(g2):  # noqa: F811
    """Pages that nobody has written hold what is not finite; a fork that took one for its source's gap would read it."""
    import torch

    rng = np.random.default_rng(0)
    page, d = 16, 64
    b = Both(g2, 8, 6, 40, page)
    b.append([0, 1, 2, 3], [70, 64, 33, 90])
    pools = [torch.full((40, 2, page, d), float("nan"), device="cuda").bfloat16() for _ in range(2)]
    for p in pools:
        p[torch.as_tensor([e for row in b.ref.table for e in row if e >= 0], device="cuda")] = torch.randn(18, 2, page, d, device="cuda").bfloat16()
    for row, i in ((0, 4), (2, 1), (3, 0), (3, 5)):  # last pages of rows 0 and 3, others in their midst
        p = b.ref.table[row][i]
        b.ref.refs[p] -= 1
        b.ref.table[row][i] = -1
    b.put()
    b.fork([0, 1, 2, 3], [7, 5, 4, 6])
    copies = g2.pages_fork(*b.dev, _int32([0, 2]), _int32([7, 4]), page=page)  # once more over itself
    b.ref.fork([0, 2], [7, 4])
    b.same()
    assert copies[0].tolist() == [-1, b.ref.table[2][2]] and copies[1].tolist() == [-1, b.ref.table[4][2]]
    g2.pages_copy(pools, *copies[:2])
    q = _dev(rng.standard_normal((2, 1, 4, d)), "bf16")
    table, lengths, _ = b.dev
    got, want = (g2.attn_decode(q, *pools, table, lengths, _int32(s)) for s in ([7, 4], [0, 2]))
    assert got.equal(want) and bool(got.isfinite().all())
    b.release([0, 1, 2, 3, 4, 5, 6, 7])
    assert not any(b.ref.refs)
