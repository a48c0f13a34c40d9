"""The 8-bit linear layer's operators (C ABI in include/dion_q8.h).

A quantized matrix is the pair Q8(data, scale): `data` [rows, cols] in
torch.float8_e4m3fn or torch.float8_e5m2, rows starting on 16-byte boundaries,
and `scale` [rows, ceil(cols / 128)] in torch.float8_e8m0fnu, one power of two
for each 1 x 128 block (or [ceil(rows / 128), ceil(cols / 128)], one for each
128 x 128 block), rows starting on 4-byte boundaries.  `new_q8` allocates one
that meets this for any size; tensors of a program's own may be passed as well.
All tensors of a call are on the current device.

The calls are the pieces of a backward pass that a program writes itself: they
have no derivative of their own.  What a call returns for inputs that require
gradients (with gradients enabled) raises in a backward pass that reaches it;
buffers that the program passed to be written carry no record.

    w8, w8t = dion_q8_quantize(W, form="both", square=True)      # weights, both orders
    x8, h, rstd = dion_rms_norm_q8(x, weight, residual=r)        # layer input
    y = dion_q8_matmul(x8, w8)                                   # y = x8 w8^T
    dy8, dy8t = dion_q8_quantize(dy, form="both")
    _, x8t = dion_q8_quantize(h, form="cols", rstd=rstd, weight=weight)
    dx = dion_q8_matmul(dy8, w8t)
    G = dion_q8_matmul(dy8t, x8t)                                # the step's gradient
    dh, dweight = dion_rms_norm_backward(dx, h, rstd, weight, dh=dh)
"""
from __future__ import annotations

import ctypes
import functools
import math
import threading
from typing import NamedTuple

import torch
from torch import empty, empty_strided

import orthonormal_optimizer_step_gb300 as _od

_E4M3, _E5M2, _E8M0 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu
_F32 = torch.float32
_ERR_WORKSPACE = _od.DION_ERR_WORKSPACE
_FORMATS = {_E4M3: 0, _E5M2: 1}
_TYPES = {torch.float32: 0, torch.bfloat16: 1}
_FORMS = {"rows": (True, False), "cols": (False, True), "both": (True, True)}
# (absent from builds of torch without CUDA, which have no tensor to call them for)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_status = {}
_status_lock = threading.Lock()


class Q8(NamedTuple):
    """A quantized matrix (or a batch of them): 8-bit values and block scales."""
    data: torch.Tensor
    scale: torch.Tensor


# Small calls are bound by the host: their checks read each attribute once, and
# the common form of an argument is recognised before a failing one is explained.
# With `stream`, a call makes it current and starts over, so that what it
# allocates comes from that stream's pool (memory that another stream's work
# still uses is then not written early).
def _type(dtype, what):
    code = _TYPES.get(dtype)
    if code is None:
        raise TypeError(f"{what} must be float32 or bfloat16, got {dtype}")
    return code


def _format(dtype):
    code = _FORMATS.get(dtype)
    if code is None:
        raise TypeError(f"8-bit format must be torch.float8_e4m3fn or torch.float8_e5m2, got {dtype}")
    return code


def _cuda(t, what):
    """The device of a CUDA tensor; it has to be the current one, where the kernels run (the default stream's handle is
    the same on every device, so a launch elsewhere would read this one's addresses)."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{what} must be a CUDA tensor")
    if dev != _current_device():
        raise ValueError(f"{what} is on cuda:{dev}, but the current device is cuda:{_current_device()}")
    return dev


def _same_device(dev, **tensors):
    for name, t in tensors.items():
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")


def _pitch(rows, cols, ld, one, what):
    """Row pitch in elements of a rows x cols matrix with strides (ld, one): its rows are contiguous and apart."""
    if cols > 1 and one != 1:
        raise ValueError(f"{what} must have contiguous rows")
    if rows <= 1 or cols == 0:
        return (cols + 15) // 16 * 16        # no second row: any pitch will do
    if ld < cols:
        raise ValueError(f"{what} must not have overlapping rows")
    return ld


def _matrix(t, what):
    """(matrix of t's rows, row pitch) of a tensor [..., cols], without a copy."""
    if t.dim() == 2:
        (_, cols), (ld, one) = t.shape, t.stride()
        if one == 1 and ld >= cols:
            return t, ld
    else:
        if t.dim() < 2:
            raise ValueError(f"{what} must have at least two dimensions")
        try:
            t = t.view(-1, t.shape[-1]) if t.numel() else t.reshape(math.prod(t.shape[:-1]), t.shape[-1])
        except RuntimeError:
            raise ValueError(f"{what} must be viewable as a matrix of rows") from None
    return t, _pitch(*t.shape, *t.stride(), what)


def _vector(t, n, what):
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous vector of {n}")


class _NoDerivative(torch.autograd.Function):
    @staticmethod
    def forward(ctx, call, outputs, *inputs):
        ctx.call = call
        return outputs

    @staticmethod
    def backward(ctx, *grads):
        raise NotImplementedError(f"{ctx.call} has no derivative: compute it with this module's calls, or detach its inputs")


def _underived(call, outputs, inputs):
    """Records that new tensors came out of `call`, so that a backward pass through them raises
    instead of stopping there; for inputs of which one requires a gradient."""
    if torch.is_grad_enabled():
        _NoDerivative.apply(call, tuple(t for t in outputs if t is not None), *inputs)


def new_q8(rows, cols, *, dtype=_E4M3, square=False, batch=None, device="cuda"):
    """An uninitialized quantized matrix (`batch` of them) with aligned rows."""
    _format(dtype)
    return _new_q8(rows, cols, dtype, square, batch, device)


def _new_q8(rows, cols, dtype, square, batch, device):
    sr, sc = (rows + 127 >> 7 if square else rows), cols + 127 >> 7
    ld, lds = cols + 15 & -16, sc + 3 & -4
    # (the allocator's sizes are multiples of 512 bytes, so a last row of scales
    # can be read to a multiple of 4 as well)
    if batch is None:
        data = (empty((rows, cols), dtype=dtype, device=device) if ld == cols else
                empty_strided((rows, cols), (ld, 1), dtype=dtype, device=device))
        scale = (empty((sr, sc), dtype=_E8M0, device=device) if lds == sc else
                 empty_strided((sr, sc), (lds, 1), dtype=_E8M0, device=device))
    else:
        data = (empty((batch, rows, cols), dtype=dtype, device=device) if ld == cols else
                empty_strided((batch, rows, cols), (rows * ld, ld, 1), dtype=dtype, device=device))
        scale = (empty((batch, sr, sc), dtype=_E8M0, device=device) if lds == sc else
                 empty_strided((batch, sr, sc), (sr * lds, lds, 1), dtype=_E8M0, device=device))
    return Q8(data, scale)


def _q8(q, what):
    """(rows, cols, format, data pitch, scale pitch, square, pointers) of a quantized matrix."""
    data, scale = q
    fmt, dptr, sptr = _FORMATS.get(data.dtype), data.data_ptr(), scale.data_ptr()
    if data.dim() == 2 == scale.dim():       # all at once; what fails is found out below
        (rows, cols), (sr, sc), (ld, one), (lds, sone) = data.shape, scale.shape, data.stride(), scale.stride()
        if (fmt is not None and scale.dtype is _E8M0 and sc == (cols + 127) >> 7 and (sr == rows or sr == (rows + 127) >> 7)
                and one == 1 == sone and ld >= cols and lds >= sc and not (ld | dptr) & 15 and not (lds | sptr) & 3):
            return rows, cols, fmt, ld, lds, sr != rows, dptr, sptr
    fmt = _format(data.dtype)
    if scale.dtype is not _E8M0:
        raise TypeError(f"{what}: scales must be torch.float8_e8m0fnu, got {scale.dtype}")
    shape, sshape, stride, sstride = data.shape, scale.shape, data.stride(), scale.stride()
    if len(shape) != len(sshape) or not 2 <= len(shape) <= 3 or shape[:-2] != sshape[:-2]:
        raise ValueError(f"{what}: {tuple(sshape)} scales do not fit {tuple(shape)} values")
    rows, cols = shape[-2], shape[-1]
    sr, sc = sshape[-2], sshape[-1]
    if sc != (cols + 127) // 128 or (sr != rows and sr != (rows + 127) // 128):
        raise ValueError(f"{what}: {tuple(sshape)} scales do not fit {tuple(shape)} values")
    ld = _pitch(rows, cols, stride[-2], stride[-1], what)
    lds = _pitch(sr, sc, sstride[-2], sstride[-1], what)
    if ld % 16 or dptr % 16:
        raise ValueError(f"{what}: rows must start on 16-byte boundaries")
    if lds % 4 or sptr % 4:
        raise ValueError(f"{what}: scale rows must start on 4-byte boundaries")
    return rows, cols, fmt, ld, lds, sr != rows, dptr, sptr


def _out_q8(q, rows, cols, dtype, square, batch, dev):
    """(data pitch, scale pitch) of a quantized matrix that a call is to write."""
    _, _, _, ld, lds, _, _, _ = _q8(q, "out")
    shape = (rows, cols) if batch is None else (batch, rows, cols)
    if tuple(q.data.shape) != shape or q.data.dtype is not dtype or q.scale.shape[-2] != ((rows + 127) // 128 if square else rows):
        raise ValueError("out does not have the shape, dtype and scales asked for")
    _same_device(dev, out=q.data, out_scale=q.scale)
    return ld, lds


# ---- status word of the products
def _status_word(dev):
    with _status_lock:                             # one word a device, whichever thread comes first
        if dev not in _status:
            # what a capture allocates and clears belongs to its graph, and it cannot be waited for
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("the first dion_q8_matmul on a device sets up its status word; make it before any stream capture")
            t = torch.zeros(1, dtype=torch.int32, device=torch.device("cuda", dev))
            torch.cuda.current_stream(dev).synchronize()   # once: later calls may run on any stream
            _status[dev] = (t.data_ptr(), t)
        return _status[dev]


def dion_q8_status(device=None) -> int:
    """Status word of dion_q8_matmul on a device (synchronize first): 0, or 4
    once any of its calls gave up waiting (their results are undefined)."""
    dev = torch.device("cuda" if device is None else device).index
    w = _status.get(torch.cuda.current_device() if dev is None else dev)
    return 0 if w is None else int(w[1].item())


# ---- operators
_NO_Q8 = (None, 0, 0, None, 0, 0)


def _q8_args(out, rows, cols, dtype, square, batch, dev, device):
    """The quantized matrix to write (a new one if `out` is None) and its arguments."""
    if out is None:
        out = _new_q8(rows, cols, dtype, square, batch, device)
        ld, lds = cols + 15 & -16, (cols + 127 >> 7) + 3 & -4
    else:
        ld, lds = _out_q8(out, rows, cols, dtype, square, batch, dev)
    data, scale = out
    if batch is None:
        return out, (data.data_ptr(), ld, 0, scale.data_ptr(), lds, 0)
    return out, (data.data_ptr(), ld, data.stride(0), scale.data_ptr(), lds, scale.stride(0))


def dion_q8_quantize(x, *, form="rows", square=False, dtype=_E4M3, rstd=None, weight=None, out=None, stream=None):
    """Quantizes x [rows, cols] or [batch, rows, cols] (float32 or bfloat16).

    form "rows": x with blocks along its rows; "cols": its transpose, with blocks
    down x's columns; "both": the two from one read.  Returns (rows, cols), each
    a Q8 or None.  square: one scale for each 128 x 128 block.  With rstd [rows]
    and weight [cols], x * rstd * weight is quantized instead of x.  out: the
    pair (rows, cols) to write into."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return dion_q8_quantize(x, form=form, square=square, dtype=dtype, rstd=rstd, weight=weight, out=out)
    wanted = _FORMS.get(form)
    if wanted is None:
        raise ValueError(f"form must be 'rows', 'cols' or 'both', got {form!r}")
    if x.dim() == 2:
        (rows, cols), (ld, one), batch, sx = x.shape, x.stride(), None, 0
    elif x.dim() == 3:
        (batch, rows, cols), (sx, ld, one) = x.shape, x.stride()
    else:
        raise ValueError("expected a [rows, cols] or [batch, rows, cols] tensor")
    dt, fmt, dev, device = _type(x.dtype, "x"), _format(dtype), _cuda(x, "x"), x.device
    if one != 1 or ld < cols:
        ld = _pitch(rows, cols, ld, one, "x")
    wdt, rptr, wptr = 0, None, None
    if rstd is not None or weight is not None:
        if rstd is None or weight is None or batch is not None:
            raise ValueError("rstd and weight go together, with a [rows, cols] tensor")
        if rstd.dtype is not _F32:
            raise TypeError(f"rstd must be float32, got {rstd.dtype}")
        wdt = _type(weight.dtype, "weight")
        _vector(weight, cols, "weight")
        _vector(rstd, rows, "rstd")
        _same_device(dev, rstd=rstd, weight=weight)
        rptr, wptr = rstd.data_ptr(), weight.data_ptr()
    q = qt = None
    qa = qta = _NO_Q8
    if wanted[0]:
        q, qa = _q8_args(None if out is None else out[0], rows, cols, dtype, square, batch, dev, device)
    if wanted[1]:
        qt, qta = _q8_args(None if out is None else out[1], cols, rows, dtype, square, batch, dev, device)
    if rows and cols and batch != 0:
        code = _od.lib().dion_q8_quantize(1 if batch is None else batch, rows, cols, dt, x.data_ptr(), ld, sx, rptr, wptr,
                                          wdt, square, fmt, *qa, *qta, _raw_stream(dev))
        if code:
            _od._check(code, "dion_q8_quantize")
    if x.requires_grad or rstd is not None and (rstd.requires_grad or weight.requires_grad):
        given = (None, None) if out is None else out
        _underived("dion_q8_quantize", [t for new, o in ((q, given[0]), (qt, given[1])) if o is None and new
                                        for t in new], (x, rstd, weight))
    return q, qt


def dion_q8_matmul(a, b, *, out=None, out_dtype=torch.bfloat16, stream=None):
    """a b^T [m, n] of quantized matrices a [m, k] and b [n, k], in float32 sums
    rounded once to out_dtype (bfloat16 or float32; that of `out` if given).

    The first call on a device sets up its status word (dion_q8_status); make it
    before any stream capture."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return dion_q8_matmul(a, b, out=out, out_dtype=out_dtype)
    m, k, af, lda, ldsa, a_sq, aptr, saptr = _q8(a, "a")
    n, k2, bf, ldb, ldsb, b_sq, bptr, sbptr = _q8(b, "b")
    ad, asc = a
    bd, bsc = b
    if k != k2 or ad.dim() != 2 or bd.dim() != 2:
        raise ValueError(f"expected [m, k] and [n, k], got {tuple(ad.shape)} and {tuple(bd.shape)}")
    dev, given = _cuda(ad, "a"), out
    if out is None:
        ct, ldc = _type(out_dtype, "out_dtype"), n
        out = empty((m, n), dtype=out_dtype, device=ad.device)
    else:
        if out.shape != (m, n):
            raise ValueError(f"out must be {m} x {n}, got {tuple(out.shape)}")
        ct, ldc = _type(out.dtype, "out"), _pitch(m, n, *out.stride(), "out")
    if not dev == asc.get_device() == bd.get_device() == bsc.get_device() == out.get_device():
        _same_device(dev, a_scale=asc, b=bd, b_scale=bsc, out=out)
    code = _od.lib().dion_q8_matmul(m, n, k, aptr, lda, af, saptr, ldsa, a_sq, bptr, ldb, bf, sbptr, ldsb, b_sq,
                                    out.data_ptr(), ldc, ct, (_status.get(dev) or _status_word(dev))[0], _raw_stream(dev))
    if code:
        _od._check(code, "dion_q8_matmul")
    if given is None and (ad.requires_grad or bd.requires_grad):
        _underived("dion_q8_matmul", (out,), (ad, bd))
    return out


def dion_rms_norm_q8(x, weight, *, residual=None, eps=1e-6, dtype=_E4M3, h=None, out=None, rstd=None, stream=None):
    """h = x + residual; the rows of h / sqrt(mean(h^2) + eps) * weight, quantized.

    x, residual [..., cols] (float32 or bfloat16), weight [cols].  Returns
    (y, h, rstd): the Q8 of all rows, the sum in x's type and shape (x itself
    without a residual; `h` may be given, also as x or residual) and
    1 / sqrt(mean(h^2) + eps) of each row, which the backward pass reads."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return dion_rms_norm_q8(x, weight, residual=residual, eps=eps, dtype=dtype, h=h, out=out, rstd=rstd)
    given = h, out, rstd
    xdt, device = x.dtype, x.device
    dt, wdt, dev = _type(xdt, "x"), _type(weight.dtype, "weight"), _cuda(x, "x")
    x2, ldx = _matrix(x, "x")
    rows, cols = x2.shape
    _vector(weight, cols, "weight")
    rptr, ldr, hptr, ldh = None, 0, None, 0
    if residual is not None:
        shape = x.shape
        if residual.shape != shape or residual.dtype is not xdt:
            raise ValueError("residual must have x's shape and dtype")
        r2, ldr = _matrix(residual, "residual")
        if h is None:
            h = empty(shape, dtype=xdt, device=device)
            hptr, ldh = h.data_ptr(), cols
        else:
            if h.shape != shape or h.dtype is not xdt:
                raise ValueError("h must have x's shape and dtype")
            h2, ldh = _matrix(h, "h")
            hptr = h2.data_ptr()
        rptr = r2.data_ptr()
        if not dev == residual.get_device() == h.get_device():
            _same_device(dev, residual=residual, h=h)
    elif h is not None:
        raise ValueError("h is written only with a residual")
    if out is None:
        fmt, ldq, lds = _format(dtype), cols + 15 & -16, (cols + 127 >> 7) + 3 & -4
        out = _new_q8(rows, cols, dtype, False, None, device)
    else:
        fmt = _format(out.data.dtype)
        ldq, lds = _out_q8(out, rows, cols, out.data.dtype, False, None, dev)
    if rstd is None:
        rstd = empty((rows,), dtype=_F32, device=device)
    else:
        if rstd.dtype is not _F32:
            raise TypeError(f"rstd must be float32, got {rstd.dtype}")
        _vector(rstd, rows, "rstd")
    if not dev == weight.get_device() == rstd.get_device():
        _same_device(dev, weight=weight, rstd=rstd)
    if not cols:
        rstd.fill_(float("nan"))                   # the mean of nothing
    elif rows:
        code = _od.lib().dion_rms_norm_q8(rows, cols, dt, x2.data_ptr(), ldx, rptr, ldr, weight.data_ptr(), wdt, eps,
                                          hptr, ldh, fmt, out[0].data_ptr(), ldq, out[1].data_ptr(), lds,
                                          rstd.data_ptr(), _raw_stream(dev))
        if code:
            _od._check(code, "dion_rms_norm_q8")
    if x.requires_grad or weight.requires_grad or residual is not None and residual.requires_grad:
        _underived("dion_rms_norm_q8", (h if residual is not None and given[0] is None else None,
                                        *((None, None) if given[1] is not None else out),
                                        rstd if given[2] is None else None), (x, weight, residual))
    return out, (x if residual is None else h), rstd


@functools.lru_cache(maxsize=256)
def _backward_workspace(rows, cols, dev):
    """dion_rms_norm_backward_workspace_size on the current device, `dev` (the size follows its number of SMs)."""
    return dion_rms_norm_backward_workspace_size(rows, cols)


def dion_rms_norm_backward_workspace_size(rows: int, cols: int) -> int:
    out = ctypes.c_size_t(0)
    _od._check(_od.lib().dion_rms_norm_backward_workspace_size(rows, cols, ctypes.byref(out)),
               "dion_rms_norm_backward_workspace_size")
    return out.value


def dion_rms_norm_backward(dy, h, rstd, weight, *, dh=None, dx=None, dweight=None, workspace=None, stream=None):
    """Gradients (dx, dweight) of dion_rms_norm_q8 from dy, the gradient of its
    (unquantized) rows, and dh, that of h along the residual stream, which is
    added to dx.  dx is the gradient of both x and residual and may be dy or dh
    itself; dweight is float32."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return dion_rms_norm_backward(dy, h, rstd, weight, dh=dh, dx=dx, dweight=dweight, workspace=workspace)
    given = dx, dweight
    ydt, shape, device = dy.dtype, dy.shape, dy.device
    dt, wdt, dev = _type(ydt, "dy"), _type(weight.dtype, "weight"), _cuda(dy, "dy")
    for t in (h, dx, dh):
        if t is not None and (t.shape != shape or t.dtype is not ydt):
            raise ValueError(f"{'h' if t is h else 'dx' if t is dx else 'dh'} must have dy's shape and dtype")
    (y2, ldy), (h2, ldh) = _matrix(dy, "dy"), _matrix(h, "h")
    rows, cols = y2.shape
    dptr, lddh = None, 0
    if dh is not None:
        d2, lddh = _matrix(dh, "dh")
        dptr = d2.data_ptr()
        if dh.get_device() != dev:
            _same_device(dev, dh=dh)
    small = False
    if dx is None:
        dx = empty(shape, dtype=ydt, device=device)
        xptr, ldx = dx.data_ptr(), cols
        # the library uses no workspace then; should its limit be lower, its answer says so
        small = cols <= 8192 and rows <= 2048 and rows * cols <= 1 << 21
    else:
        x2, ldx = _matrix(dx, "dx")
        xptr = x2.data_ptr()
    _vector(weight, cols, "weight")
    if dweight is None:
        dweight = empty((cols,), dtype=_F32, device=device)
    if rstd.dtype is not _F32 or dweight.dtype is not _F32:
        raise TypeError("rstd and dweight must be float32")
    _vector(rstd, rows, "rstd")
    _vector(dweight, cols, "dweight")
    wsptr, nbytes = None, 0
    if workspace is not None:
        _same_device(dev, workspace=workspace)
        wsptr, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif not small:
        nbytes = max(256, _backward_workspace(rows, cols, dev))
        workspace = empty((nbytes,), dtype=torch.uint8, device=device)
        wsptr = workspace.data_ptr()
    if not dev == h.get_device() == rstd.get_device() == weight.get_device() == dx.get_device() == dweight.get_device():
        _same_device(dev, h=h, rstd=rstd, weight=weight, dx=dx, dweight=dweight)
    if cols:
        code = _od.lib().dion_rms_norm_backward(rows, cols, dt, y2.data_ptr(), ldy, h2.data_ptr(), ldh, rstd.data_ptr(),
                                                weight.data_ptr(), wdt, dptr, lddh, xptr, ldx, dweight.data_ptr(),
                                                wsptr, nbytes, _raw_stream(dev))
        if code == _ERR_WORKSPACE and workspace is None:      # (with a dx given, the call takes one)
            dion_rms_norm_backward(dy, h, rstd, weight, dh=dh, dx=dx, dweight=dweight)
        elif code:
            _od._check(code, "dion_rms_norm_backward")
    if dy.requires_grad or h.requires_grad or rstd.requires_grad or weight.requires_grad or dh is not None and dh.requires_grad:
        _underived("dion_rms_norm_backward", (None if given[0] is not None else dx, None if given[1] is not None else dweight),
                   (dy, h, rstd, weight, dh))
    return dx, dweight
