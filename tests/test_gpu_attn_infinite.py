"""Scores that are infinite, of keys that a token sees: -inf has no weight, and where there is nothing else the result is zero, as for a token that
sees no key; +inf makes it not finite. Rows of heads and tokens do not touch each other."""
import numpy as np
import pytest

from tests.test_gpu_attn_decode import Case
from tests.test_gpu_attn_prologue import _dev, _np, g2  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [("f32", 64, 2), ("f32", 128, 8), ("f32", 256, 3), ("bf16", 64, 2), ("bf16", 64, 8), ("bf16", 128, 2), ("bf16", 128, 8), ("bf16", 256, 2),
          ("bf16", 256, 8)]


def keys(c, first):
    """The first component of every key of the cache."""
    k = _np(c.pools[0]).copy()
    k[..., 0] = first
    c.pools[0] = _dev(k, c.dtype)


@pytest.mark.parametrize("dtype,d,G", SHAPES)
@pytest.mark.parametrize("N", [1, 4])
@pytest.mark.parametrize("first", [-np.inf, -1e30])
def test_nothing_but_minus_infinity(g2, first, N, dtype, d, G):  # noqa: F811
    """Whole rows of such scores, in one block and in parts of many; and those of every other head alone."""
    c = Case([700, 3, 20000, 16, 129], N, 2 * G, 2, d, 16, dtype, seed=G)
    keys(c, first)
    c.q[..., 0] = 1e10
    got = c.run(g2)
    assert bool((got == 0).all())
    c.q[:, :, ::2, 0] = 0.0 if first == -1e30 else -1e10  # without that component; or scores of +inf
    got = c.run(g2)
    assert bool((got[:, :, 1::2] == 0).all())
    seen = got[:, :, ::2][:, N - 1:]  # the newest token sees some keys in every row
    assert bool(seen.isfinite().all() and seen.any(-1).all()) if first == -1e30 else not bool(seen.isfinite().any())


@pytest.mark.parametrize("dtype,d,G", SHAPES)
def test_one_key_of_minus_infinity_has_no_weight(g2, dtype, d, G):  # noqa: F811
    """As if it had no page: the results with and without it."""
    c = Case([700, 65, 20000], 1, 2 * G, 2, d, 1, dtype, seed=d)
    c.q[..., 0] = 1.0
    at = {s: int(c.lengths[s]) // 2 for s in c.slots}
    for s, t in at.items():
        c.pools[0][c.table[s, t], ..., 0] = -np.inf
    got = c.run(g2)
    for s, t in at.items():
        c.table[s, t] = -1
    assert got.equal(c.run(g2)) and bool(got.isfinite().all())
