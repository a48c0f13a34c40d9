"""Forms of the norm, its gradient and the quantization that need particular
sizes, types or values to be reached, against 64 bits with the tolerances of
test_q8_gpu, and the norm's stored sum bit for bit."""
import ctypes

import numpy as np
import pytest
import torch

import orthonormal_optimizer_step_gb300 as od
from test_q8_gpu import BF16, E4M3, E5M2, F32, NORM_SIZES, STREAM_SIZES, check_backward, check_norm, randn, same_q8

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


# ------------------------------------------------------------- the norm's forms
@pytest.mark.parametrize("wdtype,fmt", [(F32, E4M3), (BF16, E5M2), (F32, E5M2)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", STREAM_SIZES)
def test_norm_streamed_types(rows, cols, residual, wdtype, fmt):
    """The streaming kernel with float32 weights and with the wider-range format."""
    x, w = randn(rows, cols, dtype=BF16, spread=0.5), (1 + 0.1 * randn(cols, seed=1)).to(wdtype)
    r = randn(rows, cols, dtype=BF16, seed=2, std=3.0) if residual else None
    got, names = launched(lambda: od.dion_rms_norm_q8(x, w, residual=r, dtype=fmt))
    assert names == {"rms_norm_q8_stream"}
    check_norm(x, r, w, 1e-6, fmt, got)


@pytest.mark.parametrize("dtype,wdtype,fmt", [(BF16, BF16, E4M3), (BF16, F32, E5M2), (F32, BF16, E4M3)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols,off", [(3, 16389, 0), (2, 33001, 0), (2, 32768, 1), (3, 16640, 3)])
def test_norm_of_long_unaligned_rows(rows, cols, off, residual, dtype, wdtype, fmt):
    base, w = randn(2, rows, cols + off, dtype=dtype, spread=0.5), (1 + 0.1 * randn(cols, seed=1)).to(wdtype)
    x, r = base[0, :, off:], base[1, :, off:] if residual else None
    got, names = launched(lambda: od.dion_rms_norm_q8(x, w, residual=r, dtype=fmt))
    assert names == {"rms_norm_q8_long"}
    check_norm(x, r, w, 1e-6, fmt, got)
    if residual:
        torch.testing.assert_close(got[1], (x.float() + r.float()).to(dtype), rtol=0, atol=0)


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


# -------------------------------------------------------- the gradient's forms
def gradient_inputs(rows, cols, dtype, wdtype, residual, off=0):
    base = [randn(rows, cols + off, dtype=dtype, seed=i, std=s)[:, off:] for i, s in ((0, 1.0), (2, 0.01), (3, 0.01))]
    w = (1 + 0.1 * randn(cols, seed=1)).to(wdtype)
    rstd = 1.0 / torch.sqrt(base[0].float().square().mean(1) + 1e-6)
    return base[1], base[0], rstd, w, base[2] if residual else None


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", [(7, 1000), (100, 768), (33, 1001)] + STREAM_SIZES)
def test_backward_of_bfloat16_rows_with_float32_weights(rows, cols, residual):
    args = gradient_inputs(rows, cols, BF16, F32, residual)
    got, names = launched(lambda: od.dion_rms_norm_backward(*args[:4], dh=args[4]))
    want = {"rms_norm_backward_stream", "rms_norm_backward_sum"} if (rows, cols) in STREAM_SIZES else {"rms_norm_backward_small"}
    assert names == want
    check_backward(*args, got, BF16)


# several rows a CTA: of one row of registers, of four chunks a thread, and longer than the registers hold
@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (F32, F32), (BF16, F32)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols,off,name", [
    (3000, 1001, 0, "rms_norm_backward"), (3000, 1004, 0, "rms_norm_backward"), (2100, 1024, 1, "rms_norm_backward"),
    (1000, 9001, 0, "rms_norm_backward"), (1000, 9004, 0, "rms_norm_backward"), (400, 16384, 3, "rms_norm_backward"),
    (400, 16389, 0, "rms_norm_backward_long"), (400, 16640, 0, "rms_norm_backward_long"),
    (310, 20000, 1, "rms_norm_backward_long")])
def test_backward_of_several_rows_a_cta(rows, cols, off, name, residual, dtype, wdtype):
    args = gradient_inputs(rows, cols, dtype, wdtype, residual, off)
    got, names = launched(lambda: od.dion_rms_norm_backward(*args[:4], dh=args[4]))
    assert names == {name, "rms_norm_backward_sum"}
    check_backward(*args, got, dtype)


# ------------------------------------------------------ quantization of h rstd w
@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("form", ["rows", "cols", "both"])
@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("rows,cols,off", [(1, 64, 0), (200, 500, 0), (129, 1024, 0), (300, 393, 1)])
def test_quantize_normed_forms(rows, cols, off, dtype, wdtype, form, square, fmt):
    """Every form, with infinities and NaN among the values, the factors and the products."""
    x, w = randn(rows, cols + off, dtype=dtype)[:, off:], (1 + 0.2 * randn(cols, seed=4)).to(wdtype)
    rstd = torch.rand(rows, device="cuda") + 0.5
    for special in (False, True):
        if special and rows > 1:
            x, inf = x.clone(), float("inf")
            x[0, 5], x[1, 6], x[2, :] = inf, -inf, float("nan")
            x[3, 3], w[7], rstd[9], rstd[10], rstd[11] = inf, 0.0, inf, 0.0, float("nan")
            x[12, 20], w[20], x[3, 7], x[14, 21], w[22] = 3e38, 4.0, inf, 1e-38, inf
            rstd[12] = 1.5
        with np.errstate(over="ignore", invalid="ignore"):
            y = (x.float().cpu().numpy() * rstd.cpu().numpy()[:, None]) * w.float().cpu().numpy()   # float32, as defined
        assert y.dtype == np.float32
        y = y.astype(np.float64)
        r, c = od.dion_q8_quantize(x, form=form, square=square, dtype=fmt, rstd=rstd, weight=w)
        if form != "cols":
            same_q8(r, y, fmt, square)
        if form != "rows":
            same_q8(c, y.T, fmt, square)
