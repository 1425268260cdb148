"""Units of one step and of the last few keys in the form of attention that keeps its products in tensor memory: their maxima and their sums pass
between warps through the same places. Reference and tolerances are those of the other decode tests."""
import numpy as np
import pytest

from tests.test_gpu_attn_decode import Case
from tests.test_gpu_attn_prologue import g2  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("G", [17, 24, 32])
@pytest.mark.parametrize("most", [128, 300])
def test_one_token_of_many_heads(g2, most, G, d):  # noqa: F811
    """Rows of up to one step (and of up to three) with one token each, which no key is hidden from: the same bits every time, and the right ones."""
    rng = np.random.default_rng(G)
    c = Case([int(n) for n in rng.integers(1, most + 1, 200)], 1, 2 * G, 2, d, 16, "bf16", seed=G + d)
    want = c.run(g2)
    c.check(want)
    for _ in range(50):
        assert want.equal(c.run(g2))
