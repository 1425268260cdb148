"""Refusals of the calls that say which rows take part in a step, in the library and in the binding (CPU only)."""
import pytest
import torch

from tests.test_abi_attn_cpu import Tensor, g2  # noqa: F401
from tests.test_abi_ssm_cpu import A, _p, g  # noqa: F401


def _append(g, table=A, slots=A, out=A, active=A, n=1, n_slots=4, n_pages=8, wide=4, page=16, every=1, tokens=None):  # noqa: F811
    return g.lib.gdn2_pages_append_active(_p(table), _p(table), _p(table), _p(slots), _p(tokens), every, _p(out), _p(active), n, n_slots, n_pages, wide, page, None)


def _fork(g, table=A, slots=A, out=A, active=A, n=1, n_slots=4, n_pages=8, wide=4, page=16, every=1, tokens=None):  # noqa: F811
    return g.lib.gdn2_pages_fork_active(_p(table), _p(table), _p(table), _p(slots), _p(slots), _p(out), _p(out), _p(out), _p(active), n, n_slots, n_pages, wide,
                                        page, None)


@pytest.mark.parametrize("call", [_append, _fork])
def test_argument_errors(g, call):  # noqa: F811
    bad, no, off = g.GDN2_ERR_INVALID_ARG, g.GDN2_ERR_UNSUPPORTED, g.GDN2_ERR_MISALIGNED
    assert call(g, n=-1) == bad and call(g, n_pages=-1) == bad and call(g, wide=0) == bad and call(g, page=0) == bad
    assert call(g, table=0) == bad and call(g, slots=0) == bad and call(g, out=0) == bad
    assert call(g, n=1 << 24) == no and call(g, n_pages=(1 << 30) - 1) == no and call(g, page=1 << 17) == no
    assert call(g, active=A + 2) == off and call(g, out=A + 1) == off and call(g, table=A + 2) == off
    assert call(g, n=0, table=0, slots=0, out=0, active=0) == g.GDN2_OK


def test_binding_refusals(g2):  # noqa: F811
    new, i32 = Tensor.on, torch.int32
    where = new(0, 2, 4, dtype=i32), new(0, 2, dtype=i32), new(0, 5, dtype=i32)
    slots, src, active = (new(0, 2, dtype=i32) for _ in range(3))
    append, fork = g2.pages_append.plain, g2.pages_fork.plain
    for exc, f in [
        (TypeError, lambda: append(*where, slots, 1, page=16, active=active.long())),
        (ValueError, lambda: append(*where, slots, 1, page=16, active=new(0, 3, dtype=i32))),
        (ValueError, lambda: append(*where, slots, 1, page=16, active=new(0, 1, 2, dtype=i32))),
        (ValueError, lambda: append(*where, slots, 1, page=16, active=new(1, 2, dtype=i32))),
        (ValueError, lambda: append(*where, slots, 1, page=16, active=slots)),  # a graph of the step would lose its rows
        (ValueError, lambda: append(*where, slots, 1, page=16, active=new(0, 4, dtype=i32)[::2])),
        (ValueError, lambda: fork(*where, src, slots, page=16, active=src)),
        (ValueError, lambda: fork(*where, src, slots, page=16, active=slots)),
    ]:
        with pytest.raises(exc):
            f()
    assert not g2.lib.calls
