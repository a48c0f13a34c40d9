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


# ------------------------------------------------------------------ gradients
def test_outputs_without_a_derivative():
    a, q, r = torch.ones(4, requires_grad=True), torch.ones(4, 8)[:, :4], torch.ones(4)
    with torch.no_grad():
        q8._underived("call", (q, None, r), (a, None))
        assert not q.requires_grad
    q8._underived("call", (q, None, r), (a, None))
    assert q.requires_grad and r.requires_grad
    with pytest.raises(NotImplementedError, match="call has no derivative"):
        (q.sum() + a.sum()).backward()


@pytest.mark.gpu
def test_no_operator_drops_a_gradient():
    def leaf(*shape):
        return torch.randn(*shape, device="cuda", requires_grad=True)

    x, r, w, rstd = torch.randn(4, 256, device="cuda"), torch.randn(4, 256, device="cuda"), torch.ones(256, device="cuda"), torch.ones(4, device="cuda")
    x8, _ = od.dion_q8_quantize(x)
    want = {"q": x8.data.view(torch.uint8), "c": od.dion_q8_matmul(x8, x8), "y": od.dion_rms_norm_q8(x, w, residual=r),
            "g": od.dion_rms_norm_backward(x, r, rstd, w)}

    def with_grad(t):
        return t.clone().requires_grad_()

    got_q = od.dion_q8_quantize(with_grad(x), form="both")
    a8 = od.Q8(with_grad(x8.data), x8.scale)
    cases = [[got_q[0].data, got_q[1].data], [od.dion_q8_matmul(a8, x8)], [od.dion_q8_matmul(x8, a8)]]
    for i in range(3):
        args = [with_grad(t) if j == i else t for j, t in enumerate((x, w, r))]
        y, h, s = od.dion_rms_norm_q8(args[0], args[1], residual=args[2])
        cases.append([y.data, h, s])
    for i in range(5):
        args = [with_grad(t) if j == i else t for j, t in enumerate((x, r, rstd, w, r))]
        cases.append(list(od.dion_rms_norm_backward(*args[:4], dh=args[4])))
    for outputs in cases:
        for t in outputs:
            with pytest.raises(NotImplementedError, match="no derivative"):
                t.float().sum().backward()
    assert torch.equal(got_q[0].data.detach().view(torch.uint8), want["q"])          # the values are what they were
    assert torch.equal(cases[1][0], want["c"]) and torch.equal(cases[3][1], want["y"][1])
    with torch.no_grad():
        assert not od.dion_q8_matmul(a8, x8).requires_grad and not od.dion_q8_quantize(leaf(4, 256))[0].data.requires_grad
    own = torch.empty(4, 4, dtype=torch.bfloat16, device="cuda")
    assert od.dion_q8_matmul(a8, x8, out=own) is own and not own.requires_grad       # a buffer of the program's
    xg = with_grad(x)
    y, h, _ = od.dion_rms_norm_q8(xg, w)
    assert h is xg                                                                   # x itself: nothing is lost on it
    assert not want["c"].requires_grad
