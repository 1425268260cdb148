"""Forks of rows of many pages, of which a call's threads take several entries each, against the bookkeeping request by request."""
import numpy as np
import pytest

from tests.test_gpu_attn_prologue import g2  # noqa: F401
from tests.test_gpu_pages import Both

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", range(4))
def test_forks_of_long_rows(g2, seed):  # noqa: F811
    """12 forks at once of 24 rows of up to 1500 pages, with free pages for the last pages of five of them, again and again."""
    rng = np.random.default_rng(seed)
    b = Both(g2, 48, 3000, 40000, 4)
    b.append(np.arange(24), rng.integers(1, 6000, 24))
    for row in range(36, 48):  # the others are held by rows of their own
        b.append([row], [4 * min(len(b.ref.free()) - 5, 2990)])
    assert len(b.ref.free()) == 5
    met = 0
    for _ in range(10):
        b.fork(rng.integers(0, 24, 12), 24 + rng.permutation(12))
        met += sum(n > 0 for n in b.ref.lengths[24:36])
    assert 50 <= met < 120
    b.release(np.arange(48))
    assert not any(b.ref.refs)
