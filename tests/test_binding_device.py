"""The binding of the step refuses tensors of a device that is not the current one."""
from types import SimpleNamespace

import pytest
import torch

import orthonormal_optimizer_step_gb300 as od


def fake(dev, *shape):
    """As much of a tensor as the binding reads before a launch."""
    return SimpleNamespace(dim=lambda: len(shape), shape=shape, dtype=torch.float32, is_contiguous=lambda: True,
                           is_cuda=dev >= 0, get_device=lambda: dev, device=f"cuda:{dev}", data_ptr=lambda: 1 << 20,
                           numel=lambda: 1 << 30)


CALLS = {
    "step": lambda X, G, M, Q, ws: od.dion_step_batched(X, G, M, Q, mu=0.9, lr=0.01, workspace=ws),
    "static": lambda X, G, M, Q, ws: od.dion_step_batched_static(X, G, M, Q, mu=0.9, lr=0.01),
    "muon": lambda X, G, M, Q, ws: od.muon_ns_batched(G, X=X, M=M, workspace=ws),
}


@pytest.mark.parametrize("name", CALLS)
def test_device_has_to_be_current(name, monkeypatch):
    launched = []
    refuse = SimpleNamespace(dion_step_batched=lambda *a: launched.append(a) or od.DION_OK,
                             dion_step_batched_static=lambda *a: launched.append(a) or od.DION_OK,
                             muon_ns_batched=lambda *a: launched.append(a) or od.DION_OK)
    monkeypatch.setattr(od, "lib", lambda: refuse)
    monkeypatch.setattr(od, "_stream_ptr", lambda s: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for one in range(4):
        t = [fake(int(i == one), 2, 64, 32) for i in range(4)]
        if name == "muon" and one == 3:
            continue                                # takes no Q
        with pytest.raises(ValueError, match="current device is cuda:0"):
            CALLS[name](*t, fake(0, 1 << 30))
    assert not launched
    CALLS[name](*(fake(0, 2, 64, 32) for _ in range(4)), fake(0, 1 << 30))
    assert len(launched) == 1
