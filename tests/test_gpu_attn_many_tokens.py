"""Attention of many tokens a row (a prompt in one call, or a piece of one behind a past), and of many heads in full precision over a long row.
Reference and tolerances are those of the other decode tests."""
import numpy as np
import pytest

from oracle import attn
from tests.test_gpu_attn_decode import Case, _check, _dense64, _reach
from tests.test_gpu_attn_prologue import _np, g2  # noqa: F401

pytestmark = pytest.mark.gpu


def check(c, got, window=0):
    want, mag = _dense64(c.q, *c.pools, c.table, c.lengths, c.slots, c.scale, window)
    _check(_np(got), want, mag, _reach(_np(c.q), _np(c.pools[0][:50]), c.scale, int(c.lengths.max()), c.dtype), c.dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,N,Hq,Hkv,d,page,window", [
    ([500, 1300, 499, 3], 500, 4, 2, 64, 16, 0),       # a prompt alone, one behind a past, one that lost its first token, one with three
    ([1000, 2500], 1000, 4, 1, 128, 64, 0),
    ([300, 17, 640], 300, 6, 2, 256, 24, 0),
    ([1100], 1100, 2, 2, 80, 32, 100),                 # windows that most of the keys lie before
    ([700, 2000], 130, 16, 2, 128, 48, 64),
    ([257, 4000], 129, 8, 1, 64, 7, 33),
])
def test_prompts(g2, lens, N, Hq, Hkv, d, page, window, dtype):  # noqa: F811
    c = Case(lens, N, Hq, Hkv, d, page, dtype, seed=N + d)
    got = c.run(g2, window=window)
    check(c, got, window)
    assert got.equal(c.run(g2, window=window))


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_later_tokens_do_not_reach_earlier_ones(g2, bad, window, dtype, d):  # noqa: F811
    """Key and value of one token of the call's are not finite: the tokens before it keep their bits, those that see it are not finite, and those that
    its window's end has passed keep theirs."""
    N = 200
    c = Case([200, 333, 1000], N, 8, 2, d, 16, dtype, seed=d)
    want = c.run(g2, window=window)
    check(c, want, window)
    for n in (0, 31, 32, 100, 127, 199):
        kept = [p.clone() for p in c.pools]
        for s in c.slots:
            t = int(c.lengths[s]) - N + n
            for p in c.pools:
                p[c.table[s, t // 16], :, t % 16] = bad
        got = c.run(g2, window=window)
        end = min(N, n + window) if window else N
        assert got[:, :n].equal(want[:, :n]) and not bool(got[:, n:end].isfinite().any()) and got[:, end:].equal(want[:, end:])
        c.pools = kept


@pytest.mark.parametrize("lens,Hq,Hkv,d", [([20011, 300], 32, 2, 256), ([30000], 16, 1, 128), ([9000, 1, 40], 64, 4, 64), ([5000], 40, 2, 192)])
def test_many_heads_in_full_precision(g2, lens, Hq, Hkv, d):  # noqa: F811
    c = Case(lens, 1, Hq, Hkv, d, 32, "f32", seed=d)
    got = c.run(g2)
    check(c, got)
    assert got.equal(c.run(g2)) and attn.visible(lens[0], 1, 0, 0) == (0, lens[0] - 1)
