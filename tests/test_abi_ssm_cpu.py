"""The C entry points of the selective state-space mixer without a GPU: bad arguments are refused on the host, in order,
before the device is touched, and empty calls need no tensors (CPU only)."""
import ctypes

import pytest

BF16, F32 = 1, 0


@pytest.fixture(scope="module")
def g():
    import __graft_entry__

    __graft_entry__._build_module().build()
    import gated_deltanet_mixer_gdn2_gb300 as mod

    return mod


def _p(v):
    return ctypes.c_void_p(v) if v else None


A = 0x10000  # a pointer that no check reads through


def _scan(g, path=0, p=A, ld=None, step=A, s0=None, off=None, B=1, T=200, H=4, G=2, P=64, N=128, dt=BF16, ws=A, wsb=1 << 40):
    lx, lb = ld or H * P, G * N
    return g.lib.gdn2_ssm_chunk_fwd(path, _p(p), lx, _p(step), _p(step), _p(p), lb, _p(p), lb, None, _p(s0), None, _p(off), _p(p),
                                    B, T, H, G, P, N, dt, _p(ws), wsb, None)


def _grad(g, path=0, p=A, ld=None, step=A, s0=None, B=1, T=200, H=4, G=2, P=64, N=128, dt=BF16, ws=A, wsb=1 << 40):
    lx, lb = H * P, G * N
    return g.lib.gdn2_ssm_backward(path, _p(p), lx, _p(step), _p(step), _p(p), lb, _p(p), lb, None, _p(s0), _p(p), ld or lx, None,
                                   None, _p(p), lx, _p(step), _p(step), _p(p), lb, _p(p), lb, None, None, B, T, H, G, P, N, dt,
                                   _p(ws), wsb, None)


@pytest.mark.parametrize("call", [_scan, _grad])
def test_scan_argument_errors(g, call):
    bad, no, off = g.GDN2_ERR_INVALID_ARG, g.GDN2_ERR_UNSUPPORTED, g.GDN2_ERR_MISALIGNED
    assert call(g, dt=7) == bad and call(g, path=9) == bad
    assert call(g, H=3) == bad                      # heads that do not divide into the groups
    assert call(g, T=-1) == bad and call(g, B=-1) == bad and call(g, G=0) == bad
    assert call(g, p=0) == bad and call(g, step=0) == bad
    assert call(g, ld=100) == bad                   # rows shorter than their contents
    assert call(g, N=24) == no and call(g, P=12) == no and call(g, P=264) == no
    assert call(g, B=65536, T=1) == no and call(g, B=4, T=1 << 28) == no
    assert call(g, path=2, dt=F32) == no and call(g, path=2, P=32) == no and call(g, path=2, N=256) == no
    assert call(g, ld=1 << 31) == no
    assert call(g, ld=4 * 64 + 4) == off            # rows off the 16-byte boundaries
    assert call(g, p=A + 8) == off and call(g, step=A + 1) == off and call(g, s0=A + 4) == off
    assert call(g, B=0, p=0, step=0) == g.GDN2_OK   # nothing to do
    assert call(g, T=0, p=0, step=0) == g.GDN2_OK


def test_scan_workspace(g):
    size = lambda f, **k: getattr(g.lib, "gdn2_ssm_%s_workspace_size" % f)(
        k.get("path", 0), k.get("B", 1), k.get("T", 4096), k.get("H", 1), k.get("G", 1), 64, k.get("N", 128), k.get("packed", 0), k.get("dt", BF16))
    assert size("chunk_fwd") > 0                          # one head: cut, with a state for every part
    assert size("chunk_fwd", B=64, H=8) == 0              # enough heads to run whole
    assert size("chunk_fwd", N=24) == 0 and size("chunk_fwd", B=0) == 0 and size("backward", T=0) == 0
    assert size("backward") > 0 and size("backward", T=8192) > size("backward")
    for call, kw in ((_scan, dict(T=4096, H=1, G=1)), (_grad, dict(T=4096, H=1, G=1))):
        assert call(g, ws=0, **kw) == g.GDN2_ERR_WORKSPACE
        assert call(g, wsb=100, **kw) == g.GDN2_ERR_WORKSPACE
        assert call(g, ws=A + 4, **kw) == g.GDN2_ERR_MISALIGNED


def _prologue(g, p=A, w=A, state=None, off=None, ld=None, ldd=None, B=1, T=8, ch=64, H=2, dt=BF16):
    return g.lib.gdn2_ssm_prologue(_p(p), ld or ch, _p(p), ldd or H, _p(w), None, _p(w), _p(w), _p(state), _p(off), _p(p), _p(p), _p(p),
                                   B, T, ch, H, 1, dt, None)


def _prologue_grad(g, p=A, w=A, state=None, off=None, ld=None, ldd=None, B=1, T=8, ch=64, H=2, dt=BF16, ws=A, wsb=1 << 30):
    return g.lib.gdn2_ssm_prologue_backward(_p(p), ld or ch, _p(p), ldd or H, _p(w), None, _p(w), _p(w), _p(off), _p(p), ch, _p(p), _p(p),
                                            _p(p), ch, _p(p), H, _p(w), None, _p(w), _p(w), B, T, ch, H, 1, dt, _p(ws), wsb, None)


@pytest.mark.parametrize("call", [_prologue, _prologue_grad])
def test_prologue_argument_errors(g, call):
    bad, no, off = g.GDN2_ERR_INVALID_ARG, g.GDN2_ERR_UNSUPPORTED, g.GDN2_ERR_MISALIGNED
    assert call(g, dt=5) == bad and call(g, H=0) == bad and call(g, ch=0) == bad and call(g, T=-1) == bad
    assert call(g, p=0) == bad and call(g, w=0) == bad and call(g, ld=63) == bad and call(g, ldd=1) == bad
    assert call(g, ch=60) == no and call(g, ch=(1 << 20) + 8) == no and call(g, H=40000) == no and call(g, B=4, T=1 << 28) == no
    assert call(g, ld=1 << 31) == no
    assert call(g, p=A + 1) == off and call(g, w=A + 4) == off and call(g, off=A + 2) == off
    # without tokens the forward has nothing to write; the parameters' gradients are sums over no rows, and are written
    assert call(g, B=0, p=0, w=0) == (g.GDN2_OK if call is _prologue else bad)


def test_prologue_gradient_workspace(g):
    assert g.lib.gdn2_ssm_prologue_backward_workspace_size(1, 8, 64, 2, 0, BF16) > 0
    assert g.lib.gdn2_ssm_prologue_backward_workspace_size(1, 8, 60, 2, 0, BF16) == 0
    assert _prologue_grad(g, ws=0) == g.GDN2_ERR_WORKSPACE and _prologue_grad(g, wsb=16) == g.GDN2_ERR_WORKSPACE


def _decode(g, p=A, w=A, st=A, slots=None, n_slots=0, ld=None, B=1, H=4, G=2, P=64, N=128, dt=BF16, sdt=F32):
    ch = H * P + 2 * G * N
    return g.lib.gdn2_ssm_decode_step(_p(p), ld or ch, _p(p), H, _p(w), None, _p(w), _p(w), None, _p(w), _p(st), sdt, _p(slots), n_slots,
                                      _p(p), B, H, G, P, N, dt, None)


def test_decode_step_argument_errors(g):
    bad, no, off = g.GDN2_ERR_INVALID_ARG, g.GDN2_ERR_UNSUPPORTED, g.GDN2_ERR_MISALIGNED
    assert _decode(g, dt=3) == bad and _decode(g, sdt=3) == bad and _decode(g, H=3) == bad and _decode(g, B=-1) == bad
    assert _decode(g, slots=A, n_slots=-1) == bad and _decode(g, ld=8) == bad
    assert _decode(g, p=0) == bad and _decode(g, w=0) == bad and _decode(g, st=0) == bad
    assert _decode(g, P=48) == no and _decode(g, N=96) == no and _decode(g, B=65536) == no
    assert _decode(g, st=A + 8) == off and _decode(g, w=A + 8) == off and _decode(g, p=A + 1) == off and _decode(g, slots=A + 2, n_slots=1) == off
    assert _decode(g, B=0, p=0, w=0, st=0) == g.GDN2_OK


def _norm(g, x=A, z=None, post=None, pre=None, r=A, n=None, rows=4, d=64, groups=1, eps=1e-5, dt=BF16):
    return g.lib.gdn2_block_norm(_p(x), _p(z), _p(post), None, None, _p(pre), _p(r), _p(n), rows, d, groups, eps, dt, None)


def _norm_grad(g, x=A, z=None, post=None, pre=None, r=A, n=None, rows=4, d=64, groups=1, eps=1e-5, dt=BF16, ws=A, wsb=1 << 30, dz=None):
    return g.lib.gdn2_block_norm_backward(_p(x), _p(z), _p(post), None, None, _p(pre), _p(r), _p(n), _p(x), _p(dz or z), _p(post), None, None,
                                          _p(pre), rows, d, groups, eps, dt, _p(ws), wsb, None)


@pytest.mark.parametrize("call", [_norm, _norm_grad])
def test_block_norm_argument_errors(g, call):
    bad, no, off = g.GDN2_ERR_INVALID_ARG, g.GDN2_ERR_UNSUPPORTED, g.GDN2_ERR_MISALIGNED
    assert call(g, dt=4) == bad and call(g, rows=-1) == bad and call(g, d=0) == bad and call(g, groups=0) == bad
    assert call(g, x=0) == bad and call(g, pre=A) == bad and call(g, n=A) == bad      # n and its weight go together
    assert call(g, groups=2) == bad                                                   # groups belong to the norm after
    assert call(g, d=60) == no and call(g, d=8200) == no and call(g, post=A, groups=3) == no
    assert call(g, x=A + 8) == off and call(g, z=A + 2) == off and call(g, post=A + 4) == off
    assert call(g, x=0, rows=0) == g.GDN2_OK


def test_block_norm_gradient_refusals(g):
    assert g.lib.gdn2_block_norm_backward_workspace_size(4, 64) > 0
    assert g.lib.gdn2_block_norm_backward_workspace_size(4, 60) == 0
    assert _norm_grad(g, ws=0) == g.GDN2_ERR_WORKSPACE and _norm_grad(g, wsb=16) == g.GDN2_ERR_WORKSPACE
    assert _norm_grad(g, dz=A) == g.GDN2_ERR_INVALID_ARG  # a gradient of an input that is not there
