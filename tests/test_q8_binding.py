"""The binding of the 8-bit operators: what it refuses or sets up before a launch."""
import threading
import time
from types import SimpleNamespace

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


# ---------------------------------------------------------------- status word
def fake_torch(made, capturing=False):
    """As much of torch as a status word takes; allocating it takes a while."""
    def zeros(*_, device, **__):
        time.sleep(0.05)
        made.append(SimpleNamespace(data_ptr=lambda n=len(made): 1000 + n))
        return made[-1]

    cuda = SimpleNamespace(is_current_stream_capturing=lambda: capturing,
                           current_stream=lambda dev: SimpleNamespace(synchronize=lambda: None))
    return SimpleNamespace(zeros=zeros, int32=None, device=lambda kind, dev: (kind, dev), cuda=cuda)


def test_threads_share_one_status_word(monkeypatch):
    made, got = [], []
    monkeypatch.setattr(q8, "torch", fake_torch(made))
    monkeypatch.setattr(q8, "_status", {})
    threads = [threading.Thread(target=lambda: got.append(q8._status_word(0)[0])) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(made) == 1 and got == [1000] * 8


def test_status_word_is_not_made_in_a_capture(monkeypatch):
    made = []
    monkeypatch.setattr(q8, "_status", {})
    monkeypatch.setattr(q8, "torch", fake_torch(made, capturing=True))
    with pytest.raises(RuntimeError, match="before any stream capture"):
        q8._status_word(0)
    assert not made and not q8._status
    monkeypatch.setattr(q8, "torch", fake_torch(made))
    word = q8._status_word(0)
    monkeypatch.setattr(q8, "torch", fake_torch(made, capturing=True))
    assert q8._status_word(0) is word and len(made) == 1


@pytest.mark.gpu
def test_first_product_in_a_capture(monkeypatch):
    a, _ = od.dion_q8_quantize(torch.randn(4, 256, device="cuda"))
    od.dion_q8_matmul(a, a)
    words = dict(q8._status)
    x = torch.zeros(8, device="cuda")
    monkeypatch.setattr(q8, "_status", {})
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x += 1
        with pytest.raises(RuntimeError, match="before any stream capture"):
            od.dion_q8_matmul(a, a)
    g.replay()                                     # the refusal left the capture as it was
    assert bool((x == 1).all())
    monkeypatch.setattr(q8, "_status", words)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = od.dion_q8_matmul(a, a)
    g.replay()
    assert torch.equal(c, od.dion_q8_matmul(a, a))
