"""The block norm where a block walks over many rows with many warps, each of its sums following another one: with the norm
after the block alone, the norm before the next block alone, and both; against the fp64 reference, and bit for bit from
call to call (a partial sum of one row that is read in another shows as a difference, if not as an error).

Tolerances as in test_gpu_ssm.py."""
import pytest

from oracle import ssm
from tests.test_gpu_ssm import TOL, _close, _dev, _norm_dev, _norm_inputs, g2  # noqa: F401

pytestmark = pytest.mark.gpu

# (gate, post, residual, scale, pre)
FORMS = {"post": (0, 1, 1, 0, 0), "post, gate": (1, 1, 0, 0, 0), "pre": (0, 0, 0, 0, 1), "pre, residual": (0, 0, 1, 0, 1),
         "post and pre": (1, 1, 1, 1, 1)}
# rows per block from 4 to 13; groups of whole warps' vectors (256 elements), of less, and two vectors per thread
SIZES = [(3000, 2048, 1), (2000, 4096, 8), (1500, 4096, 32), (700, 8192, 4)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d,groups", SIZES)
@pytest.mark.parametrize("form", FORMS, ids=lambda s: s.replace(" ", ""))
def test_many_rows_per_block(g2, dtype, rows, d, groups, form):  # noqa: F811
    import torch

    flags = FORMS[form]
    groups = groups if flags[1] else 1
    args, d_r, d_n = _norm_inputs(dtype, rows, d, flags, 61)
    dev = _norm_dev(args, dtype)
    if not flags[2] and flags[4]:
        d_r = None
    ups = [None if t is None else _dev(t, dtype) for t in (d_r, d_n)]
    forward = lambda: g2.block_norm(*dev, groups=groups)  # noqa: E731
    backward = lambda: g2.block_norm_backward(*dev, *ups, groups=groups)  # noqa: E731
    outs, grads = forward(), backward()
    for name, a, b in zip(("r", "n"), outs, ssm.block_norm(*args, groups=groups)):
        if a is not None:
            _close(name, a, b, TOL[dtype])
    want = ssm.block_norm_grad(*args, d_r, d_n, groups=groups)
    for name, a, b, given in zip(("dx", "dz", "dpost", "dresidual", "dscale", "dpre"), grads, want, args):
        if a is not None:
            _close(name, a, b, TOL["f32"] if given.ndim == 1 else TOL[dtype])
    for call, first in ((forward, outs), (backward, grads)):
        for _ in range(20):
            for a, b in zip(first, call()):
                assert a is None or torch.equal(a, b)
