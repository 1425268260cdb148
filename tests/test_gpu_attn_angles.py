"""Angles of far positions and of frequencies beyond a radian per position, against position * inv_freq modulo a turn in exact fractions; and rows
that belong to no sequence or to an inactive slot, which no result has anything of.

Tolerance of a cosine or sine: the angle's 2^-33 (1 + f / 2 pi) turns, its rounding to 24 bits of half a turn (pi 2^-25, and pi 2^-31 from the bits
that are cut off), and 2^-22 of the function."""
from decimal import Decimal, getcontext
from fractions import Fraction

import numpy as np
import pytest

from tests.test_gpu_attn_prologue import Call, _int32, g2  # noqa: F401

pytestmark = pytest.mark.gpu

PI = Fraction(Decimal("3.14159265358979323846264338327950288419716939937510582097494459"))


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("most", [1.0, 30.0, 1024.0])
def test_far_and_fast(g2, most, pairs):  # noqa: F811
    import torch

    getcontext().prec = 70
    pos = [0, 1, -1, 3, 1000, 16777217, -16777219, 2 ** 30 + 1, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, -2 ** 31 + 77]
    freq = np.float32(most) ** np.linspace(-1, 1, 8, dtype=np.float32)
    x = torch.zeros(1, len(pos), 1, 16, device="cuda")
    x[..., 0::2 if pairs else 1] = 1.0
    if not pairs:
        x[..., 8:] = 0.0
    y, _ = g2.attn_prologue(x, x, None, None, torch.from_numpy(freq).cuda(), _int32(pos)[None], interleaved=pairs)
    y = y[0, :, 0].double().cpu().numpy()
    c, s = (y[:, 0::2], y[:, 1::2]) if pairs else (y[:, :8], y[:, 8:])
    for i, p in enumerate(pos):
        for j, f in enumerate(freq):
            turns = Fraction(float(f)) * p / (2 * PI)
            angle = float((turns - round(turns)) * 2 * PI)
            off = 2 * np.pi * 2.0 ** -33 * (1 + float(f) / (2 * np.pi)) + np.pi * (2.0 ** -25 + 2.0 ** -31) + 2.0 ** -22
            assert abs(c[i, j] - np.cos(angle)) <= off and abs(s[i, j] - np.sin(angle)) <= off, (p, float(f))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_count_for_nothing(g2, dtype):  # noqa: F811
    """Rows before, behind and between hold what is not finite: results, gradients and caches are those without them."""
    import torch

    c = Call([5, 0, 12, 3], 4, 2, 64, 32, dtype, packed=True, pad=3, seed=1)
    dead = torch.ones(c.lead[0], dtype=torch.bool, device="cuda")
    for lo, hi in c.seqs:
        dead[lo:hi] = False
    table = torch.arange(16, dtype=torch.int32, device="cuda").reshape(4, 4)
    lengths, slots = _int32([5, 12, 3, 9]), _int32([0, 3, -1, 2])  # the third sequence's slot is none
    inactive = torch.zeros_like(dead)
    inactive[c.seqs[2][0]:c.seqs[2][1]] = True

    def run():
        q, k = g2.attn_prologue(c.q, c.k, c.qw, c.kw, c.freq, offsets=c.offsets)
        got = g2.attn_prologue_backward(c.q, c.k, *c.grads, c.qw, c.kw, c.freq, offsets=c.offsets)
        return [t[~dead] for t in (q, k, *got[:2])] + list(got[2:])

    def paged():
        pools = [torch.full((16, 2, 16, 64), 3.0, device="cuda").to(c.q.dtype) for _ in range(2)]
        q = g2.attn_prologue_paged(c.q, c.k, c.v, *pools, table, lengths, slots, c.qw, c.kw, c.freq, offsets=c.offsets)
        return [q[~(dead | inactive)], *pools]

    want, stored = run(), paged()
    c.row[dead] = float("nan")
    for t in c.grads:
        t[dead] = float("inf")
    assert all(a.equal(b) for a, b in zip(run(), want))
    c.row[inactive] = float("nan")
    assert all(a.equal(b) for a, b in zip(paged(), stored))
