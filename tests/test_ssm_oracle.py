"""The fp64 reference of the selective state-space mixer against closed forms and central differences (CPU)."""
import numpy as np
import pytest

from oracle import ssm


def _scan_inputs(rng, rows, H, G, P, N, B):
    r = rng.standard_normal
    return [r((rows, H, P)), rng.uniform(0.01, 1, (rows, H)), -rng.uniform(0, 1, (rows, H)), r((rows, G, N)), r((rows, G, N)),
            r(H), r((B, H, N, P))]


def _differences(f, args, which, got, rng, h=1e-6):
    """<gradient, v> against the central difference of f along a random direction v, per argument. The error of
    a central difference is O(h^2) + rounding O(eps / h): 1e-7 relative bounds both here."""
    for i, grad in zip(which, got):
        v = rng.standard_normal(args[i].shape)
        lo, hi = list(args), list(args)
        lo[i], hi[i] = args[i] - h * v, args[i] + h * v
        want = (f(*hi) - f(*lo)) / (2 * h)
        have = float((grad * v).sum())
        assert abs(have - want) <= 1e-7 * max(1.0, abs(want)) + 1e-8 * np.abs(grad * v).sum(), (i, have, want)


def test_scan_without_decay_is_linear_attention():
    rng = np.random.default_rng(0)
    x, step, g, bm, cm, d, _ = _scan_inputs(rng, 9, 2, 1, 3, 4, 1)
    y, s1 = ssm.scan(x, step, 0 * g, bm, cm, None, None, [(0, 9)])
    s = np.cumsum(bm[:, :, :, None] * (step[..., None] * x)[:, :, None, :], 0)
    np.testing.assert_allclose(y, np.einsum("tn,thnp->thp", cm[:, 0], s), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(s1[0], s[-1], rtol=1e-12, atol=1e-12)


def test_scan_full_reset_forgets():
    rng = np.random.default_rng(1)
    x, step, g, bm, cm, d, s0 = _scan_inputs(rng, 8, 2, 2, 3, 4, 1)
    g[5] = -np.inf
    y, _ = ssm.scan(x, step, g, bm, cm, d, s0, [(0, 8)])
    y2, _ = ssm.scan(x[5:], step[5:], g[5:], bm[5:], cm[5:], d, None, [(0, 3)])
    np.testing.assert_allclose(y[5:], y2, rtol=1e-12)


def test_scan_gradients_against_differences():
    rng = np.random.default_rng(2)
    seqs = [(0, 4), (4, 4), (4, 11)]
    args = _scan_inputs(rng, 11, 4, 2, 3, 5, 3)
    dy, ds1 = rng.standard_normal(args[0].shape), rng.standard_normal(args[6].shape)

    def f(x, step, g, bm, cm, d, s0):
        y, s1 = ssm.scan(x, step, g, bm, cm, d, s0, seqs)
        return (y * dy).sum() + (s1 * ds1).sum()

    _differences(f, args, range(7), ssm.scan_grad(*args, seqs, dy, ds1), rng)


@pytest.mark.parametrize("silu", [True, False])
def test_prologue_gradients_against_differences(silu):
    rng = np.random.default_rng(3)
    seqs = [(0, 2), (2, 9), (9, 9), (9, 10)]
    r = rng.standard_normal
    args = [r((10, 6)), r((10, 3)), r((6, 4)), r(6), -rng.uniform(0.5, 2, 3), r(3)]
    ups = [r((10, 6)), r((10, 3)), r((10, 3))]

    def f(*a):
        u, step, g, _ = ssm.prologue(*a, seqs, silu=silu)
        return (u * ups[0]).sum() + (step * ups[1]).sum() + (g * ups[2]).sum()

    _differences(f, args, range(6), ssm.prologue_grad(*args, *ups, seqs, silu=silu), rng)


@pytest.mark.parametrize("gate,post,residual,scale,pre", [(1, 1, 1, 1, 1), (0, 0, 1, 0, 1), (1, 1, 0, 0, 0), (0, 1, 1, 1, 0), (1, 0, 0, 1, 1)])
def test_block_norm_gradients_against_differences(gate, post, residual, scale, pre):
    rng = np.random.default_rng(4)
    r = rng.standard_normal
    have = [True, gate, post, residual, scale, pre]
    shapes = [(5, 12), (5, 12), (12,), (5, 12), (12,), (12,)]
    full = [r(s) if k else None for k, s in zip(have, shapes)]
    which = [i for i in range(6) if have[i]]
    groups = 3 if post else 1
    d_r, d_n = r((5, 12)), r((5, 12)) if pre else None

    def f(*a):
        args = [None] * 6
        for i, v in zip(which, a):
            args[i] = v
        rr, n = ssm.block_norm(*args, groups=groups)
        return (rr * d_r).sum() + (0 if n is None else (n * d_n).sum())

    got = ssm.block_norm_grad(*full, d_r, d_n, groups=groups)
    _differences(f, [full[i] for i in which], range(len(which)), [got[i] for i in which], rng)


def test_decode_continues_the_scan():
    """Tokens one by one through decode() equal the prologue and scan of all of them."""
    rng = np.random.default_rng(5)
    r = rng.standard_normal
    B, T, H, G, P, N = 2, 5, 4, 2, 3, 2
    ch = H * P + 2 * G * N
    xbc, delta = r((B, T, ch)), r((B, T, H))
    w, bias, a, db, d = r((ch, 4)), r(ch), -rng.uniform(0.5, 2, H), r(H), r(H)
    conv, st = r((B, 3, ch)), r((B, H, N, P))
    seqs = ssm.spans(B, T, None)
    u, step, g, conv1 = ssm.prologue(xbc.reshape(-1, ch), delta.reshape(-1, H), w, bias, a, db, seqs, conv)
    x, bm, cm = u[:, :H * P].reshape(-1, H, P), u[:, H * P:H * P + G * N].reshape(-1, G, N), u[:, H * P + G * N:].reshape(-1, G, N)
    y, s1 = ssm.scan(x, step, g, bm, cm, d, st, seqs)
    for t in range(T):
        yt, conv, st = ssm.decode(xbc[:, t], delta[:, t], w, bias, a, db, d, conv, st)
        np.testing.assert_allclose(yt, y.reshape(B, T, H, P)[:, t], rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(st, s1, rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(conv, conv1)
