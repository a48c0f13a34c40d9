"""The binding of the 8-bit operators: what it refuses or sets up before a launch."""
import pytest
import torch

import orthonormal_optimizer_step_gb300 as od
from orthonormal_optimizer_step_gb300 import q8


# ------------------------------------------------------------- current device
class OnDevice:
    """As much of a CUDA tensor as the device check reads."""

    def __init__(self, dev):
        self.dev = dev

    def get_device(self):
        return self.dev


def test_device_has_to_be_current(monkeypatch):
    monkeypatch.setattr(q8, "_current_device", lambda: 0)
    assert q8._cuda(OnDevice(0), "x") == 0
    with pytest.raises(ValueError, match="x is on cuda:1, but the current device is cuda:0"):
        q8._cuda(OnDevice(1), "x")
    with pytest.raises(ValueError, match="CUDA"):
        q8._cuda(OnDevice(-1), "x")


def test_workspace_size_is_kept_by_device(monkeypatch):
    sizes = iter([1024, 2048])
    monkeypatch.setattr(q8, "dion_rms_norm_backward_workspace_size", lambda rows, cols: next(sizes))
    q8._backward_workspace.cache_clear()
    try:
        assert [q8._backward_workspace(64, 256, dev) for dev in (0, 1, 0, 1)] == [1024, 2048, 1024, 2048]
    finally:
        q8._backward_workspace.cache_clear()


@pytest.mark.gpu
def test_every_operator_checks_the_device(monkeypatch):
    x, w, rstd = torch.randn(4, 256, device="cuda"), torch.ones(256, device="cuda"), torch.ones(4, device="cuda")
    a, _ = od.dion_q8_quantize(x)
    monkeypatch.setattr(q8, "_current_device", lambda: x.get_device() + 1)       # refused before any launch
    for call in (lambda: od.dion_q8_quantize(x), lambda: od.dion_q8_matmul(a, a), lambda: od.dion_rms_norm_q8(x, w),
                 lambda: od.dion_rms_norm_backward(x, x, rstd, w)):
        with pytest.raises(ValueError, match="current device"):
            call()
