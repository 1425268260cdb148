"""Norm and rotation of queries and keys on the GPU, with and without the cache, and their gradients, against the fp64 reference
(oracle/attn.py).

Tolerances, fixed from the arithmetic before any run. A result is within half a step of its type (2^-8 bf16, 2^-24 fp32, relative) of the fp32
value; that one's error counts against the terms it is a sum of, |n_a cos| + |n_b sin| <= |n_a| + |n_b|: a sum of squares over d <= 256 elements
(8 in a row, 5 joinings: 13 roundings, halved by the root), four roundings of the norm, cosine and sine within 2^-22 (an angle rounded to 2^-24
of half a turn, 2 units of the function), two of the rotation: below 2^-20. Gradients have one more such sum against their terms: 2^-19. The
weights' gradients are sums over rows and heads, of which a lane adds at most 1/16 in a row, then joins up to 500 parts: (64 + items / 16) 2^-24
of the sum of the terms, each of them within 2^-19."""
import numpy as np
import pytest

import synth
from oracle import attn

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def g2():
    import gated_deltanet_mixer_gdn2_gb300 as mod

    return mod


def _dev(a, dtype):
    return synth.to_torch(np.ascontiguousarray(a, dtype=np.float32), dtype, "cuda")


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _int32(v):
    import torch

    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def _f32(a):
    import torch

    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()


class Call:
    """Inputs of a call on the device as slices of one row, and the same numbers in fp64."""

    def __init__(self, lens, Hq, Hkv, d, rot, dtype, packed=False, norm=(True, True), pairs=False, positions=None, seed=0, pad=0, base=1e4):
        rng = np.random.default_rng(seed)
        self.lens, self.Hq, self.Hkv, self.d, self.rot, self.dtype, self.packed, self.pairs = lens, Hq, Hkv, d, rot, dtype, packed, pairs
        rows = sum(lens) + 2 * pad
        self.row = _dev(rng.standard_normal((rows, (Hq + 2 * Hkv) * d)) * np.exp(rng.uniform(-3, 3, (rows, 1))), dtype)
        self.lead = (rows,) if packed else (len(lens), lens[0])
        wide = self.row.reshape(*self.lead, (Hq + 2 * Hkv) * d)
        cut = lambda lo, H: wide[..., lo * d:(lo + H) * d].unflatten(-1, (H, d))  # noqa: E731
        self.q, self.k, self.v = cut(0, Hq), cut(Hq, Hkv), cut(Hq + Hkv, Hkv)
        self.qw, self.kw = (_f32(rng.uniform(0.5, 1.5, d)) if on else None for on in norm)
        self.freq = _f32(base ** (-np.arange(rot // 2) / max(rot // 2, 1))) if rot else None
        starts = pad + np.concatenate([[0], np.cumsum(lens)])
        self.offsets = _int32(starts) if packed else None
        self.seqs = [(int(a), int(b)) for a, b in zip(starts[:-1], starts[1:])]
        self.positions = None if positions is None else _int32(positions).reshape(self.lead)
        self.index = attn.positions_of(self.seqs, rows)
        self.pos = self.index if positions is None else np.asarray(positions).reshape(-1)
        self.flat = lambda t: _np(t).reshape(rows, t.shape[-2], d)
        self.grads = [_dev(rng.standard_normal((*self.lead, H, d)), dtype) for H in (Hq, Hkv)]

    def want(self, side, shift=None):
        """y and the size of what it is a sum of."""
        x, w = (self.q, self.qw) if side == 0 else (self.k, self.kw)
        f = np.zeros(0) if self.freq is None else _np(self.freq)
        w = None if w is None else _np(w)
        pos = self.pos if shift is None else shift
        n = attn.normed(self.flat(x), w, 1e-6)
        y = attn.rotate(n, pos, f, self.pairs)
        a, b = attn.pairs_of(self.rot, self.pairs)
        mag = np.abs(n)
        mag[..., a], mag[..., b] = mag[..., a] + mag[..., b], mag[..., a] + mag[..., b]
        return y, mag


def _close(got, want, mag, dtype, c=2.0 ** -20):
    assert got.shape == want.shape
    off = np.abs(got - want) - (HALF[dtype] * np.abs(want) * (1 + 2.0 ** -7) + c * mag + 1e-30)
    assert np.isfinite(got).all() and (off <= 0).all(), float(off.max())


SHAPES = [  # lens, Hq, Hkv, d, rot, packed
    ([1], 1, 1, 16, 16, False),
    ([5, 5], 4, 2, 64, 64, False),
    ([37], 3, 3, 80, 48, False),
    ([3, 0, 1, 70, 0], 8, 1, 128, 128, True),
    ([130, 2, 700], 5, 2, 96, 32, True),
    ([260, 260, 260], 2, 1, 256, 64, False),
    ([9], 16, 2, 256, 256, True),
    ([4000], 6, 1, 64, 0, False),
    ([0, 0], 2, 2, 64, 32, True),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_prologue(g2, shape, pairs, dtype):
    lens, Hq, Hkv, d, rot, packed = shape
    c = Call(lens, Hq, Hkv, d, rot, dtype, packed, pairs=pairs, seed=len(lens))
    q, k = g2.attn_prologue(c.q, c.k, c.qw, c.kw, c.freq, None, c.offsets, interleaved=pairs)
    assert q.shape == c.q.shape and k.shape == c.k.shape and q.is_contiguous()
    for side, got in enumerate((q, k)):
        _close(c.flat(got), *c.want(side), dtype)


@pytest.mark.parametrize("norm", [(True, False), (False, True), (False, False)])
def test_prologue_without_weights(g2, norm):
    c = Call([21], 4, 2, 64, 32, "f32", norm=norm)
    for side, got in enumerate(g2.attn_prologue(c.q, c.k, c.qw, c.kw, c.freq)):
        _close(c.flat(got), *c.want(side), "f32")


@pytest.mark.parametrize("pairs", [False, True])
def test_positions_of_any_size(g2, pairs):
    """Every 32-bit position, and frequencies from 1e-7 to 300: in fp32 the angle is exact to fp32's own functions."""
    pos = [0, 1, -1, 255, 65537, 1000003, -1000003, 2 ** 31 - 1, -2 ** 31, 123456789]
    c = Call([10], 2, 1, 64, 64, "f32", pairs=pairs, positions=pos)
    c.freq = _f32(np.geomspace(1e-7, 300, 32))
    for side, got in enumerate(g2.attn_prologue(c.q, c.k, c.qw, c.kw, c.freq, c.positions, interleaved=pairs)):
        # in fp64 the reference itself knows an angle of 2^31 * 300 to 2^-53 of it: 7e-5
        want, mag = c.want(side)
        slack = np.abs(c.pos[:, None]) * 300 * 2.0 ** -53 * np.ones((10, 1))
        assert (np.abs(c.flat(got) - want) <= 2.0 ** -24 * np.abs(want) + (2.0 ** -20 + slack[..., None]) * mag).all()
        sure = np.abs(c.pos) < 2 ** 20
        _close(c.flat(got)[sure], want[sure], mag[sure], "f32")


def test_negative_and_zero_frequencies(g2):
    c = Call([12], 1, 1, 32, 32, "f32")
    c.freq = _f32(np.concatenate([[0.0, -0.0, -1.0, 1e-42], -np.geomspace(1e-5, 10, 12)]))
    for side, got in enumerate(g2.attn_prologue(c.q, c.k, c.qw, c.kw, c.freq)):
        _close(c.flat(got), *c.want(side), "f32")


def test_what_is_not_finite_stays_in_its_head(g2):
    import torch

    c = Call([6], 3, 1, 64, 64, "f32")
    q = c.q.clone()
    want, _ = g2.attn_prologue(q, c.k, c.qw, c.kw, c.freq)
    q[0, 2, 1, 5], q[0, 4, 0, 0] = float("nan"), float("inf")
    got, _ = g2.attn_prologue(q, c.k, c.qw, c.kw, c.freq)
    keep = torch.ones(6, 3, dtype=torch.bool, device="cuda")
    keep[2, 1] = keep[4, 0] = False
    assert torch.equal(got[0][keep], want[0][keep]) and bool(got[0, 2, 1].isnan().all())
    c.freq[3] = float("inf")
    got, _ = g2.attn_prologue(c.q, c.k, c.qw, c.kw, c.freq)
    assert bool(got[..., [3, 35]].isnan().all()) and bool(got[..., [2, 34]].isfinite().all())


def test_rows_of_no_sequence(g2):
    import torch

    c = Call([30, 0, 11], 3, 2, 64, 32, "bf16", packed=True, pad=9)
    q, k = torch.full_like(c.q, 7.0).contiguous(), torch.full_like(c.k, 7.0).contiguous()
    g2.gdn2_attn_prologue(c.q, c.k, c.qw, c.kw, c.freq, q, k, None, c.offsets)
    for side, got in enumerate((q, k)):
        assert bool((got[:9] == 7).all()) and bool((got[-9:] == 7).all())
        want, mag = c.want(side)
        _close(c.flat(got)[9:-9], want[9:-9], mag[9:-9], "bf16")
    grads = [torch.full_like(t, 7.0).contiguous() for t in (c.q, c.k)]
    dqw, dkw = torch.empty_like(c.qw), torch.empty_like(c.kw)
    poisoned = [t.clone() for t in (c.q.contiguous(), c.k.contiguous(), *c.grads)]
    for t in poisoned:
        t[:9] = t[-9:] = float("nan")
    g2.gdn2_attn_prologue_backward(*poisoned, c.qw, c.kw, c.freq, *grads, dqw, dkw, None, c.offsets)
    assert bool(dqw.isfinite().all()) and bool(dkw.isfinite().all())
    for got in grads:
        assert bool((got[:9] == 7).all()) and bool((got[-9:] == 7).all()) and bool(got[9:-9].isfinite().all())


# ---- into the cache -------------------------------------------------------------------------------------------------

def _cache(rng, lengths, page, Hkv, d, dtype, spare=3, wide=None):
    """Table, lengths and pools (of numbers that no call writes) for rows of these lengths."""
    per = [-(-n // page) for n in lengths]
    order, wide = rng.permutation(sum(per) + spare), wide or max(per) + 1
    table, at = np.full((len(lengths), wide), -1), 0
    for i, n in enumerate(per):
        table[i, :n] = order[at:at + n]
        at += n
    pools = [_dev(rng.standard_normal((sum(per) + spare, Hkv, page, d)), dtype) for _ in range(2)]
    return table, pools


PAGED = [  # new tokens per row, what the rows hold already, page, packed
    ([1], [0], 16, False),
    ([1, 1, 1, 1], [0, 63, 64, 1000], 64, False),
    ([4, 4], [5, 61], 24, False),
    ([3, 0, 1, 200, 33], [0, 9, 31, 100, 7], 32, True),
    ([50, 65], [3, 0], 1, True),
    ([700], [11], 129, True),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", PAGED)
@pytest.mark.parametrize("heads", [(4, 2, 64, 32), (16, 1, 256, 64), (3, 3, 80, 80)])
def test_prologue_into_pages(g2, case, heads, dtype):
    new, past, page, packed = case
    Hq, Hkv, d, rot = heads
    rng = np.random.default_rng(sum(new))
    B, rows = len(new), len(new) + 2
    slots = rng.permutation(rows)[:B]
    held = np.full(rows, 2)
    held[slots] = np.add(new, past)
    table, pools = _cache(rng, held, page, Hkv, d, dtype)
    before = [_np(p) for p in pools]
    c = Call(new, Hq, Hkv, d, rot, dtype, packed)
    q = g2.attn_prologue_paged(c.q, c.k, c.v, *pools, _int32(table), _int32(held), _int32(slots), c.qw, c.kw, c.freq, None, c.offsets)
    number = np.concatenate([p + np.arange(n) for n, p in zip(new, past)])
    _close(c.flat(q), *c.want(0, number), dtype)
    want, mag = c.want(1, number)
    k, v = _np(pools[0]), _np(pools[1])
    seq = np.repeat(np.arange(B), new)
    at = table[slots[seq], number // page]
    _close(k[at, :, number % page], want, mag, dtype)
    np.testing.assert_array_equal(v[at, :, number % page], c.flat(c.v))
    for now, was in zip((k, v), before):  # nothing else is written
        now[at, :, number % page] = was[at, :, number % page]
        np.testing.assert_array_equal(now, was)


def test_pages_that_are_not_there(g2):
    """Inactive rows are not touched; a token without a page, or before its row's first, is not stored; positions turn, but do not place."""
    import torch

    rng = np.random.default_rng(5)
    table, pools = _cache(rng, [40, 40, 40, 40, 40], 16, 2, 64, "f32")
    table[1, 2], table[2, 2] = 1000, -5
    before = [p.clone() for p in pools]
    c = Call([4] * 5, 2, 2, 64, 64, "f32", positions=np.arange(20) * 1000)
    slots, lengths = [0, 1, 2, 9, 4], [36, 36, 36, 36, 2]  # the tokens 32-35, and -2-1 of the last row
    q = torch.full((5, 4, 2, 64), 7.0, device="cuda")
    g2.gdn2_attn_prologue_paged(c.q, c.k, c.v, *pools, _int32(table), _int32(lengths), q, _int32(slots), c.qw, c.kw, c.freq, c.positions)
    assert bool((q[3] == 7).all())
    want, mag = c.want(0)
    live = [b * 4 + t for b in (0, 1, 2, 4) for t in range(4)]
    _close(c.flat(q)[live], want[live], mag[live], "f32")
    k, _ = c.want(1)
    for pool, was, new in zip(pools, before, (k, c.flat(c.v))):
        was[table[0, 2], :, :4] = _f32(new[0:4].swapaxes(0, 1))
        was[table[4, 0], :, :2] = _f32(new[18:20].swapaxes(0, 1))
        assert (pool - was).abs().max().item() <= 2.0 ** -18 * 50
        assert int((pool != before[0 if pool is pools[0] else 1]).sum()) <= 6 * 2 * 64


def test_lengths_out_of_range(g2):
    """Clamped to what the table can name: nothing is stored past it."""
    import torch

    rng = np.random.default_rng(6)
    table, pools = _cache(rng, [32, 32], 16, 1, 64, "f32", wide=2)
    before = [p.clone() for p in pools]
    c = Call([2, 2], 1, 1, 64, 0, "f32", norm=(False, False))
    g2.attn_prologue_paged(c.q, c.k, c.v, *pools, _int32(table), _int32([2 ** 31 - 1, -2 ** 31]))
    before[0][table[0, 1], :, 14:] = c.k[0].transpose(0, 1)
    before[1][table[0, 1], :, 14:] = c.v[0].transpose(0, 1)
    assert all(torch.equal(a, b) for a, b in zip(pools, before))


# ---- gradients ------------------------------------------------------------------------------------------------------

GRADS = [
    ([1], 1, 1, 16, 16, False),
    ([5, 5], 4, 2, 64, 64, False),
    ([37], 3, 3, 80, 48, False),
    ([3, 0, 1, 700, 0], 8, 1, 128, 128, True),
    ([260, 1300], 2, 1, 256, 64, True),
    ([2000, 2000], 6, 1, 64, 0, False),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("shape", GRADS)
def test_prologue_gradients(g2, shape, pairs, dtype):
    lens, Hq, Hkv, d, rot, packed = shape
    c = Call(lens, Hq, Hkv, d, rot, dtype, packed, pairs=pairs, seed=3)
    got = g2.attn_prologue_backward(c.q, c.k, *c.grads, c.qw, c.kw, c.freq, None, c.offsets, interleaved=pairs)
    again = g2.attn_prologue_backward(c.q, c.k, *c.grads, c.qw, c.kw, c.freq, None, c.offsets, interleaved=pairs)
    assert all(a.equal(b) for a, b in zip(got, again))
    f = np.zeros(0) if c.freq is None else _np(c.freq)
    for side, (x, w, dy) in enumerate(((c.q, c.qw, c.grads[0]), (c.k, c.kw, c.grads[1]))):
        x, w, dy = c.flat(x), _np(w), c.flat(dy)
        dx, dw = attn.prologue_grad(x, w, f, c.pos, dy, interleaved=pairs)
        g = np.abs(dy)
        a, b = attn.pairs_of(rot, pairs)
        g[..., a], g[..., b] = g[..., a] + g[..., b], g[..., a] + g[..., b]
        inv = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
        xh = np.abs(x * inv)
        _close(c.flat(got[side]), dx, inv * (g * w + xh * (g * w * xh).mean(-1, keepdims=True)), dtype, 2.0 ** -19)
        terms, items = (g * xh).sum((0, 1)), dy.shape[0] * dy.shape[1]
        assert (np.abs(_np(got[2 + side]) - dw) <= ((64 + items / 16) * 2.0 ** -24 + 2.0 ** -19) * terms).all()


def test_gradients_at_given_positions(g2):
    """The opposite rotation of the same positions: gradients of a rotation without norm, turned forward again, are what came in."""
    pos = np.arange(50) * 40009 - 1000000
    c = Call([20, 30], 2, 2, 64, 64, "f32", packed=True, norm=(False, False), positions=pos, base=1e6)
    dq, dk, _, _ = g2.attn_prologue_backward(c.q, c.k, *c.grads, None, None, c.freq, c.positions, c.offsets)
    q, k = g2.attn_prologue(dq, dk, None, None, c.freq, c.positions, c.offsets)
    for got, want in zip((q, k), c.grads):  # two rotations, each within 2^-20 of the pair
        assert (got - want).abs().max().item() <= 2.0 ** -18 * want.abs().max().item()
    dx, _ = attn.prologue_grad(c.flat(c.q), None, _np(c.freq), pos, c.flat(c.grads[0]))
    assert np.abs(c.flat(dq) - dx).max() <= 2.0 ** -18 * np.abs(dx).max()


@pytest.mark.parametrize("norm", [(True, False), (False, True), (False, False)])
def test_gradients_without_weights(g2, norm):
    c = Call([33], 4, 2, 64, 32, "f32", norm=norm)
    got = g2.attn_prologue_backward(c.q, c.k, *c.grads, c.qw, c.kw, c.freq)
    assert (got[2] is not None, got[3] is not None) == norm
    for side, (x, w, dy) in enumerate(((c.q, c.qw, c.grads[0]), (c.k, c.kw, c.grads[1]))):
        dx, _ = attn.prologue_grad(c.flat(x), None if w is None else _np(w), _np(c.freq), c.pos, c.flat(dy))
        assert np.abs(c.flat(got[side]) - dx).max() <= 2.0 ** -18 * np.abs(dx).max() * 4


def test_gradients_against_differences(g2):
    """<dx, u> against the forward's own central difference, in fp32: rounding 2^-24 / h and h^2 at h = 2^-7 are both below 2e-4 of the sum
    of the terms, of some 4000 of which the roundings add as their root."""
    import torch

    c = Call([16], 2, 2, 64, 64, "f32", seed=9)
    x = torch.randn(1, 16, 2, 64, device="cuda")
    w, dy, u, h = c.qw, c.grads[0], torch.randn(1, 16, 2, 64, device="cuda"), 2.0 ** -7
    f = lambda t: (g2.attn_prologue(t, c.k, w, c.kw, c.freq)[0].double() * dy.double()).sum()  # noqa: E731
    want = (f(x + h * u) - f(x - h * u)) / (2 * h)
    dx = g2.attn_prologue_backward(x, c.k, *c.grads, w, c.kw, c.freq)[0]
    terms = (dx * u).double()
    assert abs(terms.sum() - want).item() <= 2e-4 * terms.abs().sum().item()


def test_gradients_into_slices(g2):
    """dq and dk as slices of one row's gradient; rows between them stay."""
    import torch

    c = Call([50], 4, 2, 64, 64, "bf16")
    want = g2.attn_prologue_backward(c.q, c.k, *c.grads, c.qw, c.kw, c.freq)
    row = torch.full_like(c.row, 7.0).reshape(1, 50, -1)
    dq, dk = row[..., :256].unflatten(-1, (4, 64)), row[..., 256:384].unflatten(-1, (2, 64))
    g2.gdn2_attn_prologue_backward(c.q, c.k, *c.grads, c.qw, c.kw, c.freq, dq, dk, torch.empty_like(c.qw), torch.empty_like(c.kw))
    assert torch.equal(dq, want[0]) and torch.equal(dk, want[1]) and bool((row[..., 384:] == 7).all())


def test_long_and_strided(g2):
    """Offsets past 2^31 elements: rows 600 KB apart."""
    import torch

    wide = torch.empty(9000, 300_000, dtype=torch.bfloat16, device="cuda")
    q, k = wide[:, -320:-64].unflatten(-1, (4, 64)), wide[:, -64:].unflatten(-1, (1, 64))
    q.copy_(torch.randn(9000, 4, 64, device="cuda"))
    k.copy_(torch.randn(9000, 1, 64, device="cuda"))
    c = Call([9000], 4, 1, 64, 64, "bf16", packed=True)
    got = g2.attn_prologue(q, k, c.qw, c.kw, c.freq, None, c.offsets)
    want = g2.attn_prologue(q.contiguous(), k.contiguous(), c.qw, c.kw, c.freq, None, c.offsets)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_captured_with_its_gradients(g2):
    """A graph of a forward and a backward, replayed on new inputs, beside eager calls of the same tensors."""
    import torch

    c = Call([70], 4, 2, 64, 64, "bf16")
    f = lambda: (*g2.attn_prologue(c.q, c.k, c.qw, c.kw, c.freq), *g2.attn_prologue_backward(c.q, c.k, *c.grads, c.qw, c.kw, c.freq))  # noqa: E731
    f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = f()
    for _ in range(3):
        c.row.copy_(torch.randn_like(c.row))
        want = f()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
