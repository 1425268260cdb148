"""The state-space binding on more than one device, with stand-ins for tensors and library (CPU only): workspace sizes are those of the
device they are asked for on, and a call whose tensors lie elsewhere than on the current device is refused before anything is
launched."""
import types

import pytest
import torch


@pytest.fixture()
def g2(monkeypatch):
    import __graft_entry__

    __graft_entry__._build_module().build()
    import gated_deltanet_mixer_gdn2_gb300 as mod

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    mod._size_of.cache_clear()
    yield mod
    mod._size_of.cache_clear()


class Tensor:
    """As much of a tensor as the binding asks for."""

    def __init__(self, dev, *shape, dtype=torch.float32):
        self.dev, self.shape, self.dtype, self.is_cuda = dev, torch.Size(shape), dtype, dev >= 0

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000

    def numel(self):
        return self.shape.numel()


def test_workspace_sizes_belong_to_a_device(g2, monkeypatch):
    sizes, asked = iter((100, 250)), []
    monkeypatch.setattr(g2, "lib", types.SimpleNamespace(f=lambda *a: asked.append(a) or next(sizes)))
    assert g2._size_of("f", 0, 5, 6) == 100 and g2._size_of("f", 1, 5, 6) == 250
    assert g2._size_of("f", 0, 5, 6) == 100 and g2._size_of("f", 1, 5, 6) == 250
    assert asked == [(5, 6), (5, 6)]  # once per device, by the sizes alone


def test_tensors_off_the_current_device_are_refused(g2, monkeypatch):
    launched = []
    monkeypatch.setattr(g2, "lib", types.SimpleNamespace(gdn2_block_norm=lambda *a: launched.append(a) or 0))
    norm = lambda x, w, n: g2.gdn2_block_norm(Tensor(x, 4, 64), None, None, None, None, Tensor(w, 64), None, Tensor(n, 4, 64))  # noqa: E731
    norm(0, 0, 0)
    assert len(launched) == 1
    for devices in ((1, 1, 1), (0, 1, 0), (0, 0, 1), (-1, -1, -1), (0, -1, 0)):
        with pytest.raises(ValueError):
            norm(*devices)
    assert len(launched) == 1
