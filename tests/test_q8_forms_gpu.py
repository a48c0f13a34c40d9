"""Forms of the norm, its gradient and the quantization that need particular
sizes, types or values to be reached, against 64 bits with the tolerances of
test_q8_gpu, and the norm's stored sum bit for bit."""
import ctypes

import pytest
import torch

import orthonormal_optimizer_step_gb300 as od
from test_q8_gpu import BF16, E4M3, E5M2, F32, NORM_SIZES, STREAM_SIZES, check_backward, randn

pytestmark = pytest.mark.gpu


def launched(call):
    """The call's result and the names of the kernels it launched."""
    with od.profile() as p:
        got = call()
    torch.cuda.synchronize()
    return got, set(p.read())


# ------------------------------------------------------ the norm's stored sum
def special_sums(x, r):
    """Puts values into x and r whose sum is not finite, zero, or rounds at a tie."""
    inf, nan = float("inf"), float("nan")
    for i, (a, b) in enumerate([(inf, 1.0), (1.0, -inf), (inf, -inf), (nan, 2.0), (3.3e38, 3.3e38), (-0.0, 0.0),
                                (-0.0, -0.0), (1.0, 2.0 ** -8), (1.0, 3 * 2.0 ** -8), (1e-40, -1e-40), (256.0, 1.0)]):
        n = x.numel()
        at = (i * 7919) % n
        x.view(-1)[at], r.view(-1)[at] = a, b


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("special", [False, True])
@pytest.mark.parametrize("rows,cols", NORM_SIZES + STREAM_SIZES)
def test_norm_stores_the_rounded_sum(rows, cols, special, dtype):
    x, r, w = randn(rows, cols, dtype=dtype), randn(rows, cols, dtype=dtype, seed=2, std=3.0), randn(cols, seed=1)
    if special:
        special_sums(x, r)
    want = (x.float() + r.float()).to(dtype)
    _, h, _ = od.dion_rms_norm_q8(x, w, residual=r)
    torch.testing.assert_close(h, want, rtol=0, atol=0, equal_nan=True)
    assert torch.equal(torch.signbit(h)[~torch.isnan(h)], torch.signbit(want)[~torch.isnan(want)])


@pytest.mark.parametrize("residual", [False, True])
def test_norm_of_rows_without_columns(residual):
    x, w = torch.empty(7, 0, device="cuda"), torch.empty(0, device="cuda")
    q, h, rstd = od.dion_rms_norm_q8(x, w, residual=x if residual else None, rstd=torch.full((7,), 5.0, device="cuda"))
    assert q.data.shape == h.shape == (7, 0) and bool(torch.isnan(rstd).all())      # the mean of nothing
    dx, dw = od.dion_rms_norm_backward(x, x, rstd, w)
    assert dx.shape == (7, 0) and dw.shape == (0,)


# ----------------------------------------------------- the gradient's workspace
def backward_without_workspace(dy, h, rstd, w, dx, dw):
    """The C entry, float32, no workspace: its status."""
    rows, cols = dy.shape
    return od.lib().dion_rms_norm_backward(rows, cols, 0, dy.data_ptr(), dy.stride(0), h.data_ptr(), h.stride(0),
                                           rstd.data_ptr(), w.data_ptr(), 0, None, 0, dx.data_ptr(), dx.stride(0),
                                           dw.data_ptr(), None, ctypes.c_size_t(0), torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("order", [(0, 1, 2), (2, 0, 1), (1, 2, 0)])
@pytest.mark.parametrize("rows,cols,gap", [(1, 64, 0), (40, 96, 0), (40, 99, 1), (300, 256, 4)])
def test_backward_between_the_rows_of_its_inputs(rows, cols, gap, order):
    """dx, dy and h as columns of one matrix: apart, so no workspace is needed."""
    base = randn(rows, 3 * (cols + gap))
    dy, h, dx = (base[:, o * (cols + gap):o * (cols + gap) + cols] for o in order)
    rstd, w, dw = torch.rand(rows, device="cuda") + 0.5, 1 + 0.1 * randn(cols, seed=1), torch.empty(cols, device="cuda")
    before = base.clone()
    assert backward_without_workspace(dy, h, rstd, w, dx, dw) == od.DION_OK
    check_backward(dy, h, rstd, w, None, (dx, dw), F32)
    dx.copy_(before[:, order[2] * (cols + gap):order[2] * (cols + gap) + cols])
    assert torch.equal(base, before)


def test_backward_over_its_inputs_needs_a_workspace():
    rows, cols = 40, 96
    base, rstd, w, dw = randn(rows + 1, 300), torch.rand(rows, device="cuda"), randn(cols), torch.empty(cols, device="cuda")
    dy, h = base[:rows, :cols], base[:rows, 200:296]
    wide = randn(rows, 400)
    for dx in (dy, h, base[1:, :cols], base[:rows, 95:191], base[:rows, 105:201], base[1:, 200:296], base[:rows, 201:297]):
        assert backward_without_workspace(dy, h, rstd, w, dx, dw) == od.DION_ERR_WORKSPACE
        assert backward_without_workspace(h, dy, rstd, w, dx, dw) == od.DION_ERR_WORKSPACE
    # another pitch over the same addresses
    other = base.view(-1)[:rows * 301 - 5].as_strided((rows - 1, cols), (301, 1))
    assert backward_without_workspace(dy[:-1], h[:-1], rstd[:-1], w, other, dw) == od.DION_ERR_WORKSPACE
    assert backward_without_workspace(dy, h, rstd, w, wide[:, 8:104], dw) == od.DION_OK


class LowerLimit:
    """The library with a one-launch limit below the binding's."""

    def __init__(self, lib):
        self.lib, self.refused = lib, 0

    def __getattr__(self, name):
        return getattr(self.lib, name)

    def dion_rms_norm_backward(self, *args):
        if args[-3] is None:
            self.refused += 1
            return od.DION_ERR_WORKSPACE
        return self.lib.dion_rms_norm_backward(*args)


def test_binding_follows_the_librarys_limit(monkeypatch):
    dy, h, w, rstd = randn(50, 96), randn(50, 96, seed=1), randn(96, seed=2), torch.rand(50, device="cuda") + 0.5
    lower = LowerLimit(od.lib())
    monkeypatch.setattr(od, "lib", lambda: lower)
    got = od.dion_rms_norm_backward(dy, h, rstd, w)
    assert lower.refused == 1
    check_backward(dy, h, rstd, w, None, got, F32)
    with pytest.raises(od.DionError):              # a workspace of the caller's is not replaced
        od.dion_rms_norm_backward(dy, h, rstd, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
