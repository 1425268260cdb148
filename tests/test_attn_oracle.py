"""The fp64 reference of the attention layers' operators against closed forms and central differences (CPU)."""
import numpy as np
import pytest

from oracle import attn


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_one_and_relative(interleaved):
    """Lengths stay, the opposite rotation undoes it, and products of two rotated vectors go by the distance alone."""
    rng = np.random.default_rng(0)
    x, y = rng.standard_normal((2, 5, 3, 32))
    freq = 10.0 ** -np.arange(8)
    pos = np.array([0, 1, 7, -3, 100])
    r = attn.rotate(x, pos, freq, interleaved)
    np.testing.assert_allclose((r * r).sum(-1), (x * x).sum(-1), rtol=1e-12)
    np.testing.assert_allclose(attn.rotate(r, pos, freq, interleaved, back=True), x, rtol=0, atol=1e-12)
    np.testing.assert_array_equal(r[..., 16:], x[..., 16:])
    np.testing.assert_array_equal(r[0], x[0])
    near = (attn.rotate(x, pos, freq, interleaved) * attn.rotate(y, pos + 9, freq, interleaved)).sum(-1)
    far = (attn.rotate(x, pos + 1000, freq, interleaved) * attn.rotate(y, pos + 1009, freq, interleaved)).sum(-1)
    np.testing.assert_allclose(near, far, rtol=0, atol=1e-9)


def test_rotation_by_a_quarter():
    """A quarter turn takes (a, b) to (-b, a)."""
    x = np.arange(16.0).reshape(1, 1, 16)
    y = attn.rotate(x, np.array([1]), np.full(8, np.pi / 2), False)
    np.testing.assert_allclose(y[0, 0], np.concatenate([-x[0, 0, 8:], x[0, 0, :8]]), atol=1e-12)
    y = attn.rotate(x, np.array([1]), np.full(8, np.pi / 2), True)
    np.testing.assert_allclose(y[0, 0, 0::2], -x[0, 0, 1::2], atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_prologue_gradients(interleaved, weighted):
    """Against central differences: O(h^2) + O(eps / h) are below 1e-7 relative at h = 1e-6."""
    rng = np.random.default_rng(1)
    x, dy, w = rng.standard_normal((4, 2, 16)), rng.standard_normal((4, 2, 16)), rng.standard_normal(16) if weighted else None
    freq, pos, h = rng.uniform(0, 1, 4), np.array([0, 1, 2, 50]), 1e-6
    loss = lambda x, w: (attn.prologue(x, w, freq, pos, interleaved=interleaved) * dy).sum()  # noqa: E731
    dx, dw = attn.prologue_grad(x, w, freq, pos, dy, interleaved=interleaved)
    v = rng.standard_normal(x.shape)
    want = (loss(x + h * v, w) - loss(x - h * v, w)) / (2 * h)
    assert abs((dx * v).sum() - want) <= 1e-7 * np.abs(dx * v).sum()
    if weighted:
        v = rng.standard_normal(16)
        want = (loss(x, w + h * v) - loss(x, w - h * v)) / (2 * h)
        assert abs((dw * v).sum() - want) <= 1e-7 * np.abs(dw * v).sum()
    else:
        assert dw is None


def test_attend_of_equal_scores_is_the_mean():
    rng = np.random.default_rng(2)
    k, v = np.zeros((6, 2, 4, 16)), rng.standard_normal((6, 2, 4, 16))
    table, lengths = np.array([[5, 0, 3], [1, -1, 2]]), np.array([9, 12])
    q = rng.standard_normal((2, 1, 4, 16))
    o, _ = attn.attend(q, k, v, table, lengths, None, 1.0)
    whole = np.concatenate([v[5], v[0], v[3, :, :1]], 1)
    np.testing.assert_allclose(o[0, 0], np.repeat(whole.mean(1), 2, 0), rtol=1e-12)
    holed = np.concatenate([v[1], v[2]], 1)  # the second page is missing
    np.testing.assert_allclose(o[1, 0], np.repeat(holed.mean(1), 2, 0), rtol=1e-12)
    o, _ = attn.attend(q, k, v, table, lengths, np.array([0, 7]), 1.0, window=3)
    np.testing.assert_allclose(o[0, 0], np.repeat(whole[:, -3:].mean(1), 2, 0), rtol=1e-12)
    assert np.isnan(o[1]).all()


def test_attend_tokens_see_their_past():
    """N tokens at once are each one alone with a shorter row; tokens before the row's first see nothing."""
    rng = np.random.default_rng(3)
    k, v, q = rng.standard_normal((4, 1, 4, 16)), rng.standard_normal((4, 1, 4, 16)), rng.standard_normal((1, 4, 2, 16))
    table = np.array([[2, 1, 0, 3]])
    o, _ = attn.attend(q, k, v, table, np.array([11]), None, 0.25)
    for n in range(4):
        alone, _ = attn.attend(q[:, n:n + 1], k, v, table, np.array([8 + n]), None, 0.25)
        np.testing.assert_allclose(o[:, n:n + 1], alone, rtol=1e-12)
    o, _ = attn.attend(q, k, v, table, np.array([2]), None, 0.25)
    assert (o[0, :2] == 0).all() and (o[0, 2:] != 0).any()
    np.testing.assert_allclose(o[0, 2], np.repeat(v[2, :, :1].reshape(1, 16), 2, 0), rtol=1e-12)


def test_pages_hold_together():
    """However rows are made, forked and given back, a page's count is the number of its entries, and no row writes a shared page."""
    rng = np.random.default_rng(4)
    p = attn.Pages(np.full((6, 5), -1), np.zeros(6), np.zeros(14), 4)
    for _ in range(300):
        kind, a = rng.integers(3), rng.permutation(6)
        if kind == 0:
            p.append(a[:3], rng.integers(0, 6, 3))
        elif kind == 1:
            p.fork(a[:2], a[2:4])
        else:
            p.release(a[:1])
        entries = [e for row in p.table for e in row if e >= 0]
        assert p.refs == [entries.count(i) for i in range(14)]
        for row, n in zip(p.table, p.lengths):
            assert [e >= 0 for e in row] == [i * 4 < n for i in range(5)]
            if n % 4:
                assert p.refs[row[n // 4]] == 1
