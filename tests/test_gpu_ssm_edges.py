"""The selective state-space operators where their inputs are unusual but allowed: packed buffers with rows of no sequence,
groups of many heads, gates that are not finite or reset the state again and again.

Tolerances as in test_gpu_ssm.py, and for the same reasons: a result's own rounding and a handful of 2^-24 roundings per
term. Where a test looks at a part of a result only (the tokens behind resets), it is held to the same bound of that part's
largest value: nothing in the arithmetic of these tokens depends on what the resets have wiped out."""
import numpy as np
import pytest

from oracle import max_rel_err, ssm
from tests.test_gpu_ssm import TOL, Scan, _close, _dev, _f32, _np, _prologue_inputs, g2  # noqa: F401

pytestmark = pytest.mark.gpu

NAMES = ("dx", "dstep", "dg", "dbm", "dcm")


def _int32(v):
    import torch

    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---- rows of no sequence: before the first offset and behind the last one --------------------------------

FRONT, BACK = 7, 90
PADDED = [130, 0, 1, 40]  # lengths of the sequences between them


def _padded(a, fill, dtype):
    """Rows of `fill` around the sequences' rows."""
    a = np.asarray(a)
    return _dev(np.concatenate([np.full((n, *a.shape[1:]), fill) if n else a for n in (FRONT, 0, BACK)]), dtype)


def _padded_offsets():
    return _int32([FRONT + v for v in np.concatenate([[0], np.cumsum(PADDED)]).tolist()])


def _untouched(name, t, canary=7.0):
    assert bool((t[:FRONT] == canary).all()) and bool((t[-BACK:] == canary).all()), name


def _canvas(like, *shape):
    import torch

    return torch.full(shape or like.shape, 7.0, dtype=like.dtype, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prologue_leaves_rows_of_no_sequence(g2, dtype):  # noqa: F811
    ch, H = 136, 5
    p = _prologue_inputs(dtype, PADDED, ch, H, 71)
    seqs = ssm.spans(0, 0, np.concatenate([[0], np.cumsum(PADDED)]))
    row, off = _padded(p["row"], np.nan, dtype), _padded_offsets()
    u, step, g = _canvas(row, len(row), ch), _canvas(row, len(row), H), _canvas(row, len(row), H)
    conv = _f32(p["conv"])
    g2.gdn2_ssm_prologue(row[:, :ch], row[:, ch:ch + H], *(_f32(p[k]) for k in ("w", "bias", "a", "db")), u, step, g, conv, off)
    want = ssm.prologue(p["row"][:, :ch], p["row"][:, ch:ch + H], p["w"], p["bias"], p["a"], p["db"], seqs, p["conv"])
    for name, t, r in zip(("u", "step", "g"), (u, step, g), want):
        _untouched(name, t)
        _close(name, t[FRONT:-BACK], r, TOL[dtype])
    assert np.array_equal(_np(conv), want[3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prologue_gradients_leave_rows_of_no_sequence(g2, dtype):  # noqa: F811
    """NaN in the rows of no sequence reaches no sum over the rows, and nothing is written there."""
    ch, H = 136, 5
    p = _prologue_inputs(dtype, PADDED, ch, H, 72)
    seqs = ssm.spans(0, 0, np.concatenate([[0], np.cumsum(PADDED)]))
    row, off = _padded(p["row"], np.nan, dtype), _padded_offsets()
    par = [_f32(p[k]) for k in ("w", "bias", "a", "db")]
    dxbc, ddelta = _canvas(row, len(row), ch), _canvas(row, len(row), H)
    sums = [_canvas(t) for t in par]
    g2.gdn2_ssm_prologue_backward(row[:, :ch], row[:, ch:ch + H], *par, *(_padded(p[k], np.nan, dtype) for k in ("du", "dstep", "dg")),
                                  dxbc, ddelta, *sums, off)
    want = ssm.prologue_grad(p["row"][:, :ch], p["row"][:, ch:ch + H], p["w"], p["bias"], p["a"], p["db"], p["du"], p["dstep"],
                             p["dg"], seqs)
    for name, t, r in zip(("dxbc", "ddelta"), (dxbc, ddelta), want):
        _untouched(name, t)
        _close(name, t[FRONT:-BACK], r, TOL[dtype])
    for name, t, r in zip(("dweight", "dbias", "da", "ddelta_bias"), sums, want[2:]):
        _close(name, t, r, TOL["f32"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,G", [(6, 1), (3, 3)], ids=["heads shared out", "a head per group"])
def test_scan_leaves_rows_of_no_sequence(g2, dtype, H, G):  # noqa: F811
    import torch

    c = Scan(dtype, PADDED, True, H, G, 64, 128, seed=73)
    off = _padded_offsets()
    row = _padded(c.row, np.nan, dtype)
    x, bm, cm = (t.unflatten(-1, s) for t, s in zip(row.split([H * 64, G * 128, G * 128], -1), ((H, 64), (G, 128), (G, 128))))
    step, g, dy = (_padded(t, np.nan, dtype) for t in (c.step, c.g, c.dy))
    y, s1 = _canvas(x), torch.empty(4, H, 128, 64, device="cuda")
    g2.gdn2_ssm_chunk_fwd(x, step, g, bm, cm, y, _f32(c.d), _f32(c.s0), s1, off)
    ry, rs = c.ref()
    _untouched("y", y)
    _close("y", y[FRONT:-BACK], ry, TOL[dtype])
    _close("state", s1, rs, TOL["f32"])
    outs = [_canvas(t) for t in (x, step, g, bm, cm)]
    dd, ds0 = torch.empty(H, device="cuda"), torch.empty_like(s1)
    need = g2.lib.gdn2_ssm_backward_workspace_size(0, 4, len(row), H, G, 64, 128, 1, g2._dtype_code(x))
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")  # NaN wherever it is read before it is written
    g2.gdn2_ssm_backward(x, step, g, bm, cm, dy, *outs, dd, _f32(c.d), _f32(c.s0), _f32(c.ds1), ds0, off, workspace=ws)
    want = c.ref_grad()
    for name, t, r in zip(NAMES, outs, want):
        _untouched(name, t)
        _close(name, t[FRONT:-BACK], r, TOL[dtype])
    _close("dd", dd, want[5], TOL["f32"])
    _close("ds0", ds0, want[6], TOL["f32"])


# ---- more heads in a group than a block has threads -------------------------------------------------------

def test_skip_gradient_of_many_heads(g2):  # noqa: F811
    """Packed, 320 heads of one group, and tokens enough for a block to take all of them: dd is sum(x dy) per head, whatever the
    workspace held."""
    import torch

    c = Scan("f32", [11000, 0, 3], True, 320, 1, 8, 16, seed=74, states=False)
    x, step, g, bm, cm = c.device()
    need = g2.lib.gdn2_ssm_backward_workspace_size(0, 3, c.rows, 320, 1, 8, 16, 1, g2.GDN2_F32)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(t) for t in (x, step, g, bm, cm)]
    dd = torch.empty(320, device="cuda")
    g2.gdn2_ssm_backward(x, step, g, bm, cm, _dev(c.dy, "f32"), *outs, dd, _f32(c.d), offsets=c.offsets(), workspace=ws)
    _close("dd", dd, (c.x * c.dy).sum((0, 2)), TOL["f32"])
    assert all(bool(torch.isfinite(t).all()) for t in outs)


# ---- gates -------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("path", ["auto", "simt"])
@pytest.mark.parametrize("reset", [-np.inf, -40.0])
def test_gradients_behind_resets(g2, dtype, path, reset):  # noqa: F811
    """Ordinary decays behind many resets keep their digits: the tokens behind them are held to the bound on their own."""
    c = Scan(dtype, [32, 32], False, 2, 1, 64, 64, seed=75, decay=0.5)
    c.g = c.g.reshape(2, 32, 2)
    c.g[:, :20] = reset
    c.g = c.g.reshape(64, 2)
    got, want = c.run_grad(g2, path=path), c.ref_grad()
    for name, a, b in zip(NAMES, got, want):
        a, b = _np(a), c.lead(b)
        assert np.isfinite(a).all(), name
        e = max_rel_err(a[:, 20:], b[:, 20:])
        assert e <= TOL[dtype], (name, e)
    _close("ds0", got[6], want[6], TOL["f32"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [0, 40, 131])
def test_gate_that_is_nan(g2, dtype, at):  # noqa: F811
    """A NaN gate is no reset: what the recurrence takes through it is not finite; another head, another sequence keeps every bit."""
    import torch

    lens, H = [60, 140, 33], 3
    c = Scan(dtype, lens, True, H, H, 64, 128, seed=76)
    y, s1 = c.run(g2)
    grads = c.run_grad(g2)
    t = lens[0] + at
    c.g[t, 1] = np.nan
    yb, sb = c.run(g2)
    gb = c.run_grad(g2)
    end = lens[0] + lens[1]
    none = lambda v: not bool(torch.isfinite(v).any())  # noqa: E731
    assert none(yb[t:end, 1]) and none(sb[1, 1])
    dx, dstep, dg, dbm, dcm, _, ds0 = gb
    assert none(dx[lens[0]:t, 1]) and none(dstep[lens[0]:t, 1]) and none(dbm[lens[0]:t, 1]) and none(dcm[t:end, 1])
    assert none(dg[t:t + 1, 1]) and none(ds0[1, 1])
    keep = np.r_[0:lens[0], end:sum(lens)]
    for a, b in zip((y, *grads[:5]), (yb, *gb[:5])):
        assert torch.equal(a[keep], b[keep]) and torch.equal(a[:, [0, 2]], b[:, [0, 2]])
    for a, b in ((s1, sb), (grads[6], ds0)):
        assert torch.equal(a[[0, 2]], b[[0, 2]]) and torch.equal(a[1, [0, 2]], b[1, [0, 2]])


def test_decode_gate_that_is_nan(g2):  # noqa: F811
    import torch

    torch.manual_seed(0)
    B, H, P, N = 2, 3, 16, 32
    ch = H * P + 2 * N
    f = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    a = -f(H).abs()
    a[1] = float("nan")
    conv, st = f(B, 3, ch), f(B, H, N, P)
    y = g2.ssm_decode_step(f(B, ch), f(B, H), f(ch, 4), None, a, f(H), None, conv, st)
    assert not bool(torch.isfinite(y[:, 1]).any()) and not bool(torch.isfinite(st[:, 1]).any())
    assert bool(torch.isfinite(y[:, [0, 2]]).all()) and bool(torch.isfinite(st[:, [0, 2]]).all())
