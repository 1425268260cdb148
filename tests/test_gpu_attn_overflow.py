"""Products of queries and keys that are finite, but not when scaled: scores of +inf in every form of attention."""
import pytest

from tests.test_gpu_attn_decode import Case
from tests.test_gpu_attn_infinite import SHAPES
from tests.test_gpu_attn_prologue import g2  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d,G", SHAPES)
@pytest.mark.parametrize("N", [1, 4])
def test_scores_that_scaling_takes_to_infinity(g2, N, dtype, d, G):  # noqa: F811
    """A product of 2^127 in one head, times log2 e past the range: not finite, like any score of +inf, and the other heads keep their bits."""
    c = Case([700, 65, 20000], N, 2 * G, 2, d, 16, dtype, seed=d)
    c.scale = 1.5
    c.q.mul_(2.0 ** -6)
    c.q[..., 0] = 0.0
    want = c.run(g2)
    for s in c.slots:
        c.pools[0][c.table[s, 0], :, 0, 0] = 2.0 ** 63
    assert c.run(g2).equal(want)
    c.q[:, :, 1, 0] = 2.0 ** 64
    got = c.run(g2)
    assert not bool(got[:, :, 1].isfinite().any())
    keep = [h for h in range(2 * G) if h != 1]
    assert got[:, :, keep].equal(want[:, :, keep])
