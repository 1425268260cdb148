"""Rows without a visible key whose outputs are as large as a call admits: zeros, every one of them."""
import pytest

from tests.test_gpu_attn_prologue import _int32, g2  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wide", [4, 200])
@pytest.mark.parametrize("N,Hq,Hkv,d,dtype", [
    (4096, 512, 512, 256, "float32"),    # 2^29 elements: 2^31 bytes
    (4095, 1024, 1024, 256, "float32"),  # a row whose bytes, modulo 2^32, are not a negative number
    (4096, 4096, 4096, 64, "bfloat16"),  # 2^30 elements
])
def test_rows_of_billions_of_bytes(g2, N, Hq, Hkv, d, dtype, wide):  # noqa: F811
    import torch

    dtype = getattr(torch, dtype)
    q = torch.zeros(1, N, Hq, d, dtype=dtype, device="cuda")
    o = torch.full_like(q, 7.0)
    pools = [torch.zeros(2, Hkv, 16, d, dtype=dtype, device="cuda") for _ in range(2)]
    table = torch.zeros(1, wide, dtype=torch.int32, device="cuda")
    g2.gdn2_attn_decode(q, *pools, table, _int32([0]), o)
    assert not bool(o.any())
