"""Serving weights in 4 bits (C ABI in include/dion_q4.h).

A 4-bit matrix is Q4(data, scale, cols, group): `data` uint8 [rows, 64 *
ceil(cols / 128)] in the layout that include/dion_q4.h states, rows starting on
16-byte boundaries, and `scale` bfloat16 [rows, ceil(cols / group)], one for each
32, 64 or 128 values of a row.  All tensors of a call are on the current device.
The products are for serving: they have no derivative, and a backward pass that
reaches their results raises.

    w4 = dion_q4_quantize(W, group=128)                          # once, after training
    x8, h, rstd = dion_rms_norm_q8(x, weight, residual=r)        # a few rows
    y = dion_q4_matmul(x8, w4)                                   # or plain rows: dion_q4_matmul(x, w4)
"""
from __future__ import annotations

from typing import NamedTuple

import torch
from torch import empty

import orthonormal_optimizer_step_gb300 as _od
from orthonormal_optimizer_step_gb300.q8 import (_TYPES, Q8, _cuda, _matrix, _pitch, _q8, _raw_stream, _same_device, _type,
                                                 _underived)

_BF16, _U8 = torch.bfloat16, torch.uint8
_GROUPS = (32, 64, 128)


class Q4(NamedTuple):
    """A 4-bit matrix: held rows, group scales, columns and the group's size."""
    data: torch.Tensor
    scale: torch.Tensor
    cols: int
    group: int


def new_q4(rows, cols, *, group=128, device="cuda"):
    """An uninitialized 4-bit matrix, its scale rows on 16-byte boundaries."""
    if group not in _GROUPS:
        raise ValueError(f"group must be 32, 64 or 128, got {group!r}")
    groups = -(-cols // group)
    lds = groups + 7 & -8
    scale = (empty((rows, groups), dtype=_BF16, device=device) if lds == groups else
             torch.empty_strided((rows, groups), (lds, 1), dtype=_BF16, device=device))
    return Q4(empty((rows, (cols + 127 >> 7) * 64), dtype=torch.uint8, device=device), scale, cols, group)


def _q4(w, what):
    """(rows, cols, group, data pointer, pitch, scale pointer, pitch) of a 4-bit matrix."""
    data, scale, cols, group = w
    if data.dim() == 2 == scale.dim() and group in _GROUPS:       # all at once; what fails is found out below
        (rows, width), (sr, sc), (ldq, one), (lds, sone), qptr = data.shape, scale.shape, data.stride(), scale.stride(), data.data_ptr()
        if (one == 1 == sone and sr == rows and width == (cols + 127 >> 7) * 64 and sc * group - cols < group and sc * group >= cols > 0
                and ldq >= width and lds >= sc and not (ldq | qptr) & 15 and data.dtype is _U8 and scale.dtype is _BF16):
            return rows, cols, group, qptr, ldq, scale.data_ptr(), lds
    if group not in _GROUPS:
        raise ValueError(f"{what}: group must be 32, 64 or 128, got {group!r}")
    if data.dtype is not _U8 or scale.dtype is not _BF16:
        raise TypeError(f"{what}: data must be uint8 and scales bfloat16, got {data.dtype} and {scale.dtype}")
    if data.dim() != 2 or scale.dim() != 2 or cols < 0:
        raise ValueError(f"{what}: expected [rows, bytes] data and [rows, groups] scales")
    (rows, width), (sr, sc), (ldq, one), (lds, sone) = data.shape, scale.shape, data.stride(), scale.stride()
    if width != (cols + 127 >> 7) * 64 or sr != rows or sc != -(-cols // group):
        raise ValueError(f"{what}: {tuple(data.shape)} data and {tuple(scale.shape)} scales do not fit {cols} columns in groups of {group}")
    if one != 1 or ldq < width or rows == 1 or width == 0:
        ldq = _pitch(rows, width, ldq, one, what)
    if sone != 1 or lds < sc:
        lds = _pitch(sr, sc, lds, sone, f"{what}'s scales")
    qptr = data.data_ptr()
    if (ldq | qptr) & 15:
        raise ValueError(f"{what}: rows must start on 16-byte boundaries")
    return rows, cols, group, qptr, ldq, scale.data_ptr(), lds


def dion_q4_quantize(x, *, group=128, out=None, stream=None):
    """x [rows, cols] (float32 or bfloat16) in 4 bits: scale = bfloat16(amax / 7) of each group,
    values x / scale rounded to whole numbers -8..7."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return dion_q4_quantize(x, group=group, out=out)
    if x.dim() != 2:
        raise ValueError("expected a [rows, cols] tensor")
    (rows, cols), (ld, one) = x.shape, x.stride()
    dt, dev, given = _type(x.dtype, "x"), _cuda(x, "x"), out
    if one != 1 or ld < cols:
        ld = _pitch(rows, cols, ld, one, "x")
    if out is None:
        out = new_q4(rows, cols, group=group, device=x.device)
    r, c, g, qptr, ldq, sptr, lds = _q4(out, "out")
    if (r, c, g) != (rows, cols, group):
        raise ValueError(f"out is {r} x {c} in groups of {g}, expected {rows} x {cols} in groups of {group}")
    _same_device(dev, out=out.data, out_scale=out.scale)
    code = _od.lib().dion_q4_quantize(rows, cols, group, dt, x.data_ptr(), ld, qptr, ldq, sptr, lds, _raw_stream(dev))
    if code:
        _od._check(code, "dion_q4_quantize")
    if given is None and x.requires_grad:
        _underived("dion_q4_quantize", out[:2], (x,))
    return out


def dion_q4_dequantize(w, *, out=None, out_dtype=_BF16, stream=None):
    """The values [rows, cols] of a 4-bit matrix, rounded once to out_dtype (that of `out` if given)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return dion_q4_dequantize(w, out=out, out_dtype=out_dtype)
    rows, cols, group, qptr, ldq, sptr, lds = _q4(w, "w")
    dev = _cuda(w.data, "w")
    if out is None:
        dt, ld = _type(out_dtype, "out_dtype"), cols
        out = empty((rows, cols), dtype=out_dtype, device=w.data.device)
    else:
        if out.shape != (rows, cols):
            raise ValueError(f"out must be {rows} x {cols}, got {tuple(out.shape)}")
        dt, ld = _type(out.dtype, "out"), _pitch(rows, cols, *out.stride(), "out")
    _same_device(dev, w_scale=w.scale, out=out)
    code = _od.lib().dion_q4_dequantize(rows, cols, group, qptr, ldq, sptr, lds, dt, out.data_ptr(), ld, _raw_stream(dev))
    if code:
        _od._check(code, "dion_q4_dequantize")
    return out


def dion_q4_matmul(x, w, *, out=None, out_dtype=_BF16, stream=None):
    """x w^T [..., rows of w] for a few rows of x, [..., cols] of two dimensions or more in float32 or
    bfloat16, or a Q8 matrix (what dion_rms_norm_q8 returns); w a Q4.  Sums are float32, rounded once to out_dtype
    (bfloat16 or float32; that of `out` if given)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return dion_q4_matmul(x, w, out=out, out_dtype=out_dtype)
    n, cols, group, qptr, ldq, sptr, lds = _q4(w, "w")
    if type(x) is Q8:
        m, k, xt, ldx, ldsx, square, xptr, sxptr = _q8(x, "x")
        data, scale = x
        if data.dim() != 2 or (square and m > 1):
            raise ValueError("x must be an 8-bit [rows, cols] matrix with a scale for each 128 values of a row")
        xt += 2
        shape = m, n
    else:
        data, scale, sxptr, ldsx, xt = x, None, None, 0, _TYPES.get(x.dtype)
        if xt is None:
            _type(x.dtype, "x")
        if x.dim() == 2:
            (m, k), (ldx, one) = x.shape, x.stride()
            if one != 1 or ldx < k:
                ldx = _pitch(m, k, ldx, one, "x")
            shape, xptr = (m, n), x.data_ptr()
        else:
            x2, ldx = _matrix(x, "x")
            (m, k), shape, xptr = x2.shape, (*x.shape[:-1], n), x2.data_ptr()
    if k != cols:
        raise ValueError(f"x has {k} columns, w {cols}")
    dev, given = _cuda(data, "x"), out
    if out is None:
        yt, ldy = _TYPES.get(out_dtype), n
        if yt is None:
            _type(out_dtype, "out_dtype")
        out = empty(shape, dtype=out_dtype, device=data.device)
        yptr = out.data_ptr()
    else:
        if out.shape != shape:
            raise ValueError(f"out must be {shape}, got {tuple(out.shape)}")
        yt = _type(out.dtype, "out")
        y2, ldy = _matrix(out, "out")
        yptr = y2.data_ptr()
        if out.get_device() != dev:
            _same_device(dev, out=out)
    if not dev == w[0].get_device() == w[1].get_device() or scale is not None and scale.get_device() != dev:
        _same_device(dev, w=w.data, w_scale=w.scale, x_scale=scale)
    code = _od.lib().dion_q4_matmul(m, n, k, xt, xptr, ldx, sxptr, ldsx, group, qptr, ldq, sptr, lds, yt, yptr, ldy,
                                    _raw_stream(dev))
    if code:
        _od._check(code, "dion_q4_matmul")
    if given is None and data.requires_grad:
        _underived("dion_q4_matmul", (out,), (data,))
    return out
