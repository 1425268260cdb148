"""The selective state-space scan where its paths differ: bounded waits that run out, the CUDA-core kernels on shapes
that the tensor cores would take, and states that decay so slowly that one factor's rounding would add up.

Tolerances as in test_gpu_ssm.py. A decay of 1e-3 a token keeps a state for about 1600 tokens: a factor rounded to 2^-24
and used alike for each would be off by 1e-4; held with its remainder it leaves the states' own roundings, which add up to
the square root of 1600 times 2^-24 = 2.4e-6, within the fp32 bound."""
import numpy as np
import pytest

from oracle import ssm
from tests.test_gpu_ssm import TOL, Scan, _close, _dev, _f32, _r32, g2  # noqa: F401

pytestmark = pytest.mark.gpu


def _times_out(g2, call):
    import torch

    g2.gdn2_set_wait_limit(0)
    try:
        call()
        torch.cuda.synchronize()
        assert g2.gdn2_last_device_status() == g2.GDN2_ERR_TIMEOUT
    finally:
        g2.gdn2_set_wait_limit(-1)
    assert g2.gdn2_last_device_status() == g2.GDN2_OK  # read and cleared


def _check_forward(g2, c, state):
    y, s1 = c.run(g2, output_final_state=state)
    ry, rs = c.ref()
    _close("y", y, c.lead(ry), TOL["bf16"])
    if state:
        _close("state", s1, rs, TOL["f32"])
    assert g2.gdn2_last_device_status() == g2.GDN2_OK


@pytest.mark.parametrize("lens,H", [([130, 300], 4), ([2300], 1)], ids=["whole", "cut"])
@pytest.mark.parametrize("state", [True, False])
def test_scan_timeout_then_correct(g2, lens, H, state):  # noqa: F811
    c = Scan("bf16", lens, True, H, 1, 64, 128, seed=31)
    _times_out(g2, lambda: c.run(g2, output_final_state=state))
    _check_forward(g2, c, state)


def test_scan_gradients_timeout_then_correct(g2):  # noqa: F811
    c = Scan("bf16", [300, 70], True, 4, 2, 64, 128, seed=32)
    _times_out(g2, lambda: c.run_grad(g2))
    got, want = c.run_grad(g2), c.ref_grad()
    for name, a, b in zip(("dx", "dstep", "dg", "dbm", "dcm"), got, want):
        _close(name, a, b, TOL["bf16"])
    assert g2.gdn2_last_device_status() == g2.GDN2_OK


@pytest.mark.parametrize("lens,packed,H,G,P,N", [([130], False, 4, 2, 64, 128), ([5, 0, 128, 129, 300], True, 2, 1, 128, 64)])
def test_scan_on_cuda_cores(g2, lens, packed, H, G, P, N):  # noqa: F811
    c = Scan("bf16", lens, packed, H, G, P, N, seed=33)
    y, s1 = c.run(g2, path="simt")
    ry, rs = c.ref()
    _close("y", y, c.lead(ry), TOL["bf16"])
    _close("state", s1, rs, TOL["f32"])
    got, want = c.run_grad(g2, path="simt"), c.ref_grad()
    for name, a, b in zip(("dx", "dstep", "dg", "dbm", "dcm"), got, want):
        _close(name, a, c.lead(b), TOL["bf16"])
    _close("dd", got[5], want[5], TOL["f32"])
    _close("ds0", got[6], want[6], TOL["f32"])


def test_paths_refuse_what_they_cannot_run(g2):  # noqa: F811
    for args in (("f32", [16], False, 2, 1, 64, 128), ("bf16", [16], False, 2, 1, 32, 128), ("bf16", [16], False, 2, 1, 64, 32)):
        c = Scan(*args, seed=34)
        for call in (c.run, c.run_grad):
            with pytest.raises(g2.Gdn2Error) as e:
                call(g2, path="tcgen05")
            assert e.value.status == g2.GDN2_ERR_UNSUPPORTED


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_slow_decay(g2, dtype):  # noqa: F811
    c = Scan(dtype, [5000, 5000], False, 24, 2, 64, 64, seed=35)
    c.g = np.broadcast_to(_r32(-np.ldexp(1.0, -10) * (1 + np.arange(24) % 3 / 4)), c.g.shape).copy()  # exact in bf16
    y, s1 = c.run(g2)
    ry, rs = c.ref()
    _close("y", y, c.lead(ry), TOL[dtype])
    _close("state", s1, rs, TOL["f32"])
    c = Scan(dtype, [3000], False, 1, 1, 64, 64, seed=37)
    c.g[:] = -np.ldexp(1.0, -10)
    got, want = c.run_grad(g2), c.ref_grad()
    for name, a, b in zip(("dx", "dstep", "dg", "dbm", "dcm"), got, want):
        _close(name, a, c.lead(b), TOL[dtype])
    _close("ds0", got[6], want[6], TOL["f32"])


def test_decode_slow_decay(g2):  # noqa: F811
    """A few thousand single tokens with the same slow decay: the state against the fp64 recurrence."""
    import torch

    rng = np.random.default_rng(36)
    H, P, N, T = 2, 16, 16, 2500
    ch = H * P + 2 * N
    x = _r32(rng.standard_normal((T, ch)))
    w = _r32(np.tile([0.0, 0.0, 0.0, 1.0], (ch, 1)))  # the newest sample alone
    delta, bias = _r32(np.full((T, H), -1.0)), _r32(np.zeros(H))
    a = _r32([-3e-3, -2e-3])
    win, st = np.zeros((1, 3, ch)), np.zeros((1, H, N, P))
    dev = [_f32(v) for v in (w, a, bias, win, st)]
    xd, dd = _dev(x, "f32"), _dev(delta, "f32")
    for t in range(T):
        y = g2.ssm_decode_step(xd[t:t + 1], dd[t:t + 1], dev[0], None, dev[1], dev[2], None, dev[3], dev[4])
    u = x * ssm.sigmoid(x)
    step = ssm.softplus(delta)
    ry, rs = ssm.scan(u[:, :H * P].reshape(T, H, P), step, a * step, u[:, None, H * P:H * P + N], u[:, None, H * P + N:], None,
                      st, ssm.spans(1, T, None))
    _close("state", dev[4], rs, TOL["f32"])
    _close("y", y, ry[-1:], TOL["f32"])
    assert torch.equal(dev[3][0].cpu(), torch.from_numpy(x[-3:].astype(np.float32)))
