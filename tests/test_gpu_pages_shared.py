"""A row shortened into a page that its fork names too: its next tokens do not reach the fork."""
import numpy as np
import pytest

from tests.test_gpu_attn_prologue import _dev, _int32, g2  # noqa: F401
from tests.test_gpu_pages import Both
from tests.test_gpu_pages_shortened import shorten

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("length", [48, 47, 40, 32, 31, 16, 0])
def test_the_fork_keeps_its_tokens(g2, length):  # noqa: F811
    page, d = 16, 64
    rng = np.random.default_rng(length)
    b = Both(g2, 4, 6, 20, page)
    b.append([0], [48])
    pools = [_dev(rng.standard_normal((20, 2, page, d)), "bf16") for _ in range(2)]
    b.fork([0], [1])
    q = _dev(rng.standard_normal((1, 1, 4, d)), "bf16")
    table, lengths, _ = b.dev
    want = g2.attn_decode(q, *pools, table, lengths, _int32([1]))
    shorten(b, 0, length)
    b.append([0], [1])
    assert b.ref.lengths[0] == length + (length == 48)
    row = 0
    if length < 48:  # by a fork of its own, whose last page is a copy
        got = g2.pages_fork(*b.dev, _int32([0]), _int32([2]), page=page)
        b.same(*zip(got, b.ref.fork([0], [2])))
        g2.pages_copy(pools, *got[:2])
        row = 2
        b.append([2], [1])
        assert b.ref.lengths[2] == length + 1
    new = _dev(rng.standard_normal((1, 1, 4, d)), "bf16")
    g2.attn_prologue_paged(new, new[:, :, :2], new[:, :, 2:], *pools, table, lengths, _int32([row]))
    assert g2.attn_decode(q, *pools, table, lengths, _int32([1])).equal(want)
    b.release([0, 1, 2])
    assert not any(b.ref.refs)
