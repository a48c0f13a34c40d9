"""The 8-bit training example: its gradients against float32 autograd of the same
stack, and its loss under the Dion step."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "q8_training.py")


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("q8_training", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_gradients_follow_the_unquantized_stack(ex):
    """E4M3 keeps 4 significant bits, a relative rounding error of 2^-4 at most and
    about 2^-5.3 in the mean square; a gradient meets about a dozen such roundings
    in three layers, independent of each other: sqrt(12) 2^-5.3 < 0.1."""
    net = ex.Stack(3, 256, seed=1)
    x = torch.randn(512, 256, device="cuda").bfloat16()
    out, saved = net.forward(x)
    dout = torch.randn_like(out)
    dx = net.backward(dout, saved)
    X = net.X.float().requires_grad_()
    w = net.norm.clone().requires_grad_()
    xf = x.float().requires_grad_()
    r = xf
    for l in range(3):
        y = r / torch.sqrt(r.square().mean(-1, keepdim=True) + 1e-6) * w[l]
        r = r + y @ X[l].t()
    r.backward(dout.float())
    for got, want in ((out, r), (dx, xf.grad), (net.G, X.grad), (net.norm_grad, w.grad)):
        assert float((got.float() - want.detach()).norm() / want.detach().norm()) < 0.1


def test_loss_falls(ex):
    losses = ex.train(3, 512, 1024, 40)
    assert losses[-1] < 0.5 * losses[0]
