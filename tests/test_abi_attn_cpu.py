"""The C entry points of the attention layers without a GPU: bad arguments are refused on the host before the device is touched, and empty
calls need no tensors; and the binding's own refusals (CPU only)."""
import ctypes
import types

import pytest
import torch

from tests.test_abi_ssm_cpu import A, BF16, F32, _p, g  # noqa: F401


def _prologue(g, p=A, w=A, f=A, pos=None, off=None, ld=None, B=1, T=8, Hq=4, Hkv=2, d=64, rot=32, eps=1e-6, dt=BF16):  # noqa: F811
    return g.lib.gdn2_attn_prologue(_p(p), ld or Hq * d, _p(p), Hkv * d, _p(w), _p(w), _p(f), _p(pos), _p(off), _p(p), _p(p), B, T, Hq, Hkv, d,
                                    rot, 0, eps, dt, None)


def _paged(g, p=A, w=A, f=A, pos=None, off=None, ld=None, B=1, T=8, Hq=4, Hkv=2, d=64, rot=32, eps=1e-6, dt=BF16, table=A, lengths=A,  # noqa: F811
           slots=None, n_slots=1, n_pages=4, wide=4, page=16, pool=A):
    return g.lib.gdn2_attn_prologue_paged(_p(p), ld or Hq * d, _p(p), Hkv * d, _p(p), Hkv * d, _p(w), _p(w), _p(f), _p(pos), _p(off), _p(p),
                                          _p(pool), _p(pool), _p(table), _p(lengths), _p(slots), n_slots, n_pages, wide, page, B, T, Hq, Hkv,
                                          d, rot, 0, eps, dt, None)


def _grad(g, p=A, w=A, f=A, pos=None, off=None, ld=None, B=1, T=8, Hq=4, Hkv=2, d=64, rot=32, eps=1e-6, dt=BF16, dw=A, ws=A, wsb=1 << 30):  # noqa: F811
    lq, lk = Hq * d, Hkv * d
    return g.lib.gdn2_attn_prologue_backward(_p(p), ld or lq, _p(p), lk, _p(w), _p(w), _p(f), _p(pos), _p(off), _p(p), lq, _p(p), lk, _p(p), lq,
                                             _p(p), lk, _p(dw), _p(dw), B, T, Hq, Hkv, d, rot, 0, eps, dt, _p(ws), wsb, None)


@pytest.mark.parametrize("call", [_prologue, _paged, _grad])
def test_prologue_argument_errors(g, call):  # noqa: F811
    bad, no, off = g.GDN2_ERR_INVALID_ARG, g.GDN2_ERR_UNSUPPORTED, g.GDN2_ERR_MISALIGNED
    assert call(g, dt=5) == bad and call(g, Hq=0) == bad and call(g, Hkv=0) == bad and call(g, T=-1) == bad and call(g, B=-1) == bad
    assert call(g, rot=-16) == bad and call(g, rot=80) == bad and call(g, eps=-1.0) == bad and call(g, eps=float("nan")) == bad
    assert call(g, f=0) == bad and call(g, p=0) == bad and call(g, ld=255) == bad
    assert call(g, d=72, rot=16) == no and call(g, d=272) == no and call(g, rot=24) == no and call(g, Hq=5000) == no
    assert call(g, B=4, T=1 << 28) == no and call(g, ld=1 << 31) == no
    assert call(g, p=A + 8) == off and call(g, w=A + 4) == off and call(g, f=A + 2) == off and call(g, pos=A + 1) == off
    assert call(g, off=A + 2) == off and call(g, ld=4 * 64 + 4) == off
    assert call(g, f=0, rot=0, B=0, p=0, w=0, **({"dw": 0} if call is _grad else {})) == g.GDN2_OK  # nothing to do


def test_gradient_argument_errors(g):  # noqa: F811
    bad = g.GDN2_ERR_INVALID_ARG
    assert _grad(g, dw=0) == bad and _grad(g, w=0) == bad  # weights and their gradients go together
    assert _grad(g, ws=0) == g.GDN2_ERR_WORKSPACE and _grad(g, wsb=64) == g.GDN2_ERR_WORKSPACE and _grad(g, ws=A + 4) == g.GDN2_ERR_MISALIGNED
    size = g.lib.gdn2_attn_prologue_backward_workspace_size
    assert size(1, 8, 64, 0) >= 2 * 64 * 4 and size(0, 8, 64, 0) == 0 and size(1, 8, 65, 0) == 0 and size(3, 8, 64, 1) == size(1, 8, 64, 0)


def test_cache_argument_errors(g):  # noqa: F811
    bad, no, off = g.GDN2_ERR_INVALID_ARG, g.GDN2_ERR_UNSUPPORTED, g.GDN2_ERR_MISALIGNED
    for call in (_paged, _decode):
        assert call(g, table=0) == bad and call(g, lengths=0) == bad and call(g, n_slots=-1) == bad and call(g, n_pages=-1) == bad
        assert call(g, wide=0) == bad and call(g, page=0) == bad and call(g, pool=0) == bad
        assert call(g, page=65537) == no and call(g, wide=1 << 20, page=1 << 10) == no
        assert call(g, table=A + 2) == off and call(g, lengths=A + 1) == off and call(g, slots=A + 2) == off and call(g, pool=A + 8) == off


def _decode(g, q=A, ld=None, pool=A, table=A, lengths=A, slots=None, n_slots=1, n_pages=4, wide=4, page=16, o=A, B=1, N=1, Hq=4, Hkv=2, d=64,  # noqa: F811
            window=0, dt=BF16, ws=A, wsb=1 << 30):
    return g.lib.gdn2_attn_decode(_p(q), ld or Hq * d, _p(pool), _p(pool), _p(table), _p(lengths), _p(slots), n_slots, n_pages, wide, page, _p(o),
                                  B, N, Hq, Hkv, d, 0.125, window, dt, _p(ws), wsb, None)


def test_decode_argument_errors(g):  # noqa: F811
    bad, no, off = g.GDN2_ERR_INVALID_ARG, g.GDN2_ERR_UNSUPPORTED, g.GDN2_ERR_MISALIGNED
    assert _decode(g, dt=3) == bad and _decode(g, Hkv=3) == bad and _decode(g, N=-1) == bad and _decode(g, window=-1) == bad
    assert _decode(g, q=0) == bad and _decode(g, o=0) == bad and _decode(g, ld=255) == bad
    assert _decode(g, d=72) == no and _decode(g, d=272) == no and _decode(g, B=65536) == no and _decode(g, N=5000) == no
    assert _decode(g, ld=1 << 31) == no
    assert _decode(g, q=A + 8) == off and _decode(g, o=A + 4) == off and _decode(g, ld=260) == off and _decode(g, wide=999, ws=A + 8) == off
    assert _decode(g, wide=999, ws=0) == g.GDN2_ERR_WORKSPACE and _decode(g, wide=999, wsb=1000) == g.GDN2_ERR_WORKSPACE
    assert _decode(g, B=0, q=0, o=0, ws=0) == g.GDN2_OK and _decode(g, N=0, q=0, o=0, ws=0) == g.GDN2_OK
    size = g.lib.gdn2_attn_decode_workspace_size
    assert size(1, 1, 4, 2, 64, 999, 16, BF16) > 0 and size(1, 1, 4, 2, 64, 999, 16, F32) > 0 and size(0, 1, 4, 2, 64, 999, 16, BF16) == 0
    assert size(1, 1, 4, 3, 64, 999, 16, BF16) == 0 and size(1, 1, 4, 2, 64, 0, 16, BF16) == 0 and size(1, 1, 4, 2, 64, 4, 16, BF16) == 0  # short rows: no parts


def _fork(g, table=A, src=A, out=A, n=1, n_slots=4, n_pages=8, wide=4, page=16):  # noqa: F811
    return g.lib.gdn2_pages_fork(_p(table), _p(table), _p(table), _p(src), _p(src), _p(out), _p(out), _p(out), n, n_slots, n_pages, wide, page, None)


def _append(g, table=A, src=A, out=A, n=1, n_slots=4, n_pages=8, wide=4, page=16, every=1, tokens=None):  # noqa: F811
    return g.lib.gdn2_pages_append(_p(table), _p(table), _p(table), _p(src), _p(tokens), every, _p(out), n, n_slots, n_pages, wide, page, None)


def _release(g, table=A, src=A, n=1, n_slots=4, n_pages=8, wide=4):  # noqa: F811
    return g.lib.gdn2_pages_release(_p(table), _p(table), _p(table), _p(src), n, n_slots, n_pages, wide, None)


def test_pages_argument_errors(g):  # noqa: F811
    bad, no, off = g.GDN2_ERR_INVALID_ARG, g.GDN2_ERR_UNSUPPORTED, g.GDN2_ERR_MISALIGNED
    for call in (_fork, _append, _release):
        assert call(g, n=-1) == bad and call(g, n_slots=-1) == bad and call(g, n_pages=-1) == bad and call(g, wide=0) == bad
        assert call(g, table=0) == bad and call(g, src=0) == bad
        assert call(g, n=1 << 24) == no and call(g, wide=1 << 30) == no and call(g, n=1 << 20, wide=1 << 12) == no
        assert call(g, table=A + 2) == off and call(g, src=A + 1) == off
        assert call(g, n=0, table=0, src=0) == g.GDN2_OK
    for call in (_fork, _append):
        assert call(g, page=0) == bad and call(g, out=0) == bad and call(g, page=1 << 17) == no and call(g, wide=1 << 20, page=1 << 10) == no
        assert call(g, out=A + 2) == off
    assert _append(g, every=-1) == bad and _append(g, tokens=A + 2) == off


def test_copy_argument_errors(g):  # noqa: F811
    bad = g.GDN2_ERR_INVALID_ARG

    def call(ptrs=(A,), sizes=(64,), pools=1, src=A, n=1, rows=4):
        p, b = (ctypes.c_void_p * 1)(*ptrs), (ctypes.c_longlong * 1)(*sizes)
        return g.lib.gdn2_pages_copy(p, b, pools, _p(src), _p(src), n, rows, None)

    assert call(ptrs=(None,)) == bad and call(sizes=(-1,)) == bad and call(pools=-1) == bad and call(n=-1) == bad and call(rows=-1) == bad
    assert call(src=0) == bad and call(src=A + 2) == g.GDN2_ERR_MISALIGNED and call(sizes=(1 << 40,)) == g.GDN2_ERR_UNSUPPORTED
    assert call(n=0, src=0) == g.GDN2_OK and call(sizes=(0,), ptrs=(None,)) == g.GDN2_OK and call(rows=0, ptrs=(None,)) == g.GDN2_OK
    assert g.lib.gdn2_pages_copy(None, None, 0, None, None, 3, 4, None) == g.GDN2_OK


# ---- the binding ----------------------------------------------------------------------------------------------------

@pytest.fixture()
def g2(g, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    real, calls = g.lib, []
    monkeypatch.setattr(g, "lib", types.SimpleNamespace(calls=calls, **{n: (lambda *a, n=n: calls.append((n, a)) or 0) for n in g.EXPORTS
                                                                       if n.startswith(("gdn2_attn", "gdn2_pages"))}))
    g._size_of.cache_clear()
    yield g
    g._size_of.cache_clear()
    assert real is not g.lib


class Tensor(torch.Tensor):
    """A CPU tensor that says it lies on a device."""

    @staticmethod
    def on(dev, *shape, dtype=torch.bfloat16):
        t = torch.zeros(*shape, dtype=dtype).as_subclass(Tensor)
        t.dev = dev
        return t

    def get_device(self):
        return getattr(self, "dev", 0)


def test_binding_refusals(g2):  # noqa: F811
    new, i32 = Tensor.on, torch.int32
    q, k, w, f = new(0, 2, 3, 4, 64), new(0, 2, 3, 2, 64), new(0, 64, dtype=torch.float32), new(0, 16, dtype=torch.float32)
    q_out, k_out = new(0, 2, 3, 4, 64), new(0, 2, 3, 2, 64)
    call = lambda *a, **kw: g2.gdn2_attn_prologue.plain(*a, **kw)  # noqa: E731
    call(q, k, w, w, f, q_out, k_out)
    assert len(g2.lib.calls) == 1
    pools, table, lengths = (new(0, 5, 2, 16, 64), new(0, 5, 2, 16, 64)), new(0, 2, 4, dtype=i32), new(0, 2, dtype=i32)
    slots, ok = new(0, 2, dtype=i32), new(0, 2, 3, 4, 64)
    ws = new(0, 1 << 10, dtype=torch.uint8)
    g2.gdn2_attn_decode.plain(q, *pools, table, lengths, ok, slots, workspace=ws)
    assert len(g2.lib.calls) == 3  # the workspace's size is asked for too
    for exc, f_ in [
        (ValueError, lambda: call(new(1, 2, 3, 4, 64), k, w, w, f, q_out, k_out)),
        (ValueError, lambda: call(q, new(1, 2, 3, 2, 64), w, w, f, q_out, k_out)),
        (ValueError, lambda: call(q, new(0, 2, 4, 2, 64), w, w, f, q_out, k_out)),
        (TypeError, lambda: call(q, k.float(), w, w, f, q_out, k_out)),
        (TypeError, lambda: call(q, k, w.bfloat16(), w, f, q_out, k_out)),
        (ValueError, lambda: call(q, k, new(0, 32, dtype=torch.float32), w, f, q_out, k_out)),
        (ValueError, lambda: call(q, k, w, w, new(0, 4, 4, dtype=torch.float32), q_out, k_out)),
        (ValueError, lambda: call(q[0], k[0], w, w, f, q_out, k_out)),
        (TypeError, lambda: call(q, k, w, w, f, q_out, k_out, new(0, 2, 3, dtype=torch.int64))),
        (ValueError, lambda: call(q, k, w, w, f, q_out, k_out, new(0, 6, dtype=i32))),
        (ValueError, lambda: call(q, k, w, w, f, q_out.transpose(0, 1), k_out)),
        (ValueError, lambda: g2.gdn2_attn_decode.plain(q, pools[0], new(0, 4, 2, 16, 64), table, lengths, ok, slots, workspace=ws)),
        (ValueError, lambda: g2.gdn2_attn_decode.plain(q, *pools, table, new(0, 3, dtype=i32), ok, slots, workspace=ws)),
        (ValueError, lambda: g2.gdn2_attn_decode.plain(q, *pools, new(0, 3, 4, dtype=i32), new(0, 3, dtype=i32), ok, workspace=ws)),
        (ValueError, lambda: g2.gdn2_attn_decode.plain(q, *pools, table, lengths, ok, new(0, 3, dtype=i32), workspace=ws)),
        (TypeError, lambda: g2.gdn2_attn_decode.plain(q, *(p.float() for p in pools), table, lengths, ok, slots, workspace=ws)),
        (ValueError, lambda: g2.pages_copy.plain([pools[0], new(0, 4, 8)], slots, slots)),
        (ValueError, lambda: g2.pages_copy.plain([pools[0]], slots, new(0, 3, dtype=i32))),
        (TypeError, lambda: g2.pages_release.plain(table, lengths, new(0, 5, dtype=i32), slots.long())),
        (ValueError, lambda: g2.pages_release.plain(new(1, 2, 4, dtype=i32), lengths, new(0, 5, dtype=i32), slots)),
        (TypeError, lambda: g2.pages_append.plain(table, lengths, new(0, 5, dtype=i32), slots, 1.5, page=16)),
        (ValueError, lambda: g2.pages_append.plain(table, lengths, new(0, 5, dtype=i32), slots, -1, page=16)),
        (ValueError, lambda: g2.pages_append.plain(table, lengths, new(0, 5, dtype=i32), slots, 2 ** 32 + 1, page=16)),  # would wrap to 1
        (ValueError, lambda: g2.pages_append.plain(table, lengths, new(0, 5, dtype=i32), slots, 1, page=2 ** 32 + 16)),
        (ValueError, lambda: g2.pages_fork.plain(table, lengths, new(0, 5, dtype=i32), slots, slots, page=0)),
        (ValueError, lambda: g2.gdn2_attn_decode.plain(q, *pools, table, lengths, ok, slots, window=-1, workspace=ws)),
    ]:
        with pytest.raises(exc):
            f_()
    assert len(g2.lib.calls) == 3
