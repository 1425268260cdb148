"""How many roundings to bf16 a gradient of the tensor-core scan has, where the given states are most of it: short sequences.

The measure is the 2-norm of the error over that of the exact result, and its unit the error of rounding the exact result itself
to bf16. Independent roundings of the same size add up as the root of their number: the result's own and one operand's
make 1.41 units, one operand more 1.73. dx, dstep, dB and dC have one rounded operand in every term, so 1.55 (half-way); dg has
products of the two saved states, so 1.9. dD and the state's gradient are sums in fp32 (test_gpu_ssm.py)."""
import numpy as np
import pytest

import synth
from tests.test_gpu_ssm import Scan, _np, g2  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,G", [([1] * 48, 1), ([8] * 32, 4), ([40, 3, 0, 77, 25] * 3, 1), ([130, 60], 2)], ids=["1", "8", "mixed", "130"])
@pytest.mark.parametrize("N", [64, 128])
def test_gradients_with_states(g2, lens, G, N):  # noqa: F811
    c = Scan("bf16", lens, True, 8, G, 64, N, seed=81)
    got, want = c.run_grad(g2), c.ref_grad()
    assert g2.gdn2_last_device_status() == g2.GDN2_OK
    for name, limit, a, b in zip(("dx", "dstep", "dg", "dbm", "dcm"), (1.55, 1.55, 1.9, 1.55, 1.55), got, want):
        unit = np.linalg.norm(synth.round_to(b, "bf16").astype(np.float64) - b)
        off = np.linalg.norm(_np(a).reshape(b.shape) - b)
        assert off <= limit * unit, (name, off / unit)
