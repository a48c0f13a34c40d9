"""CPU-only checks of the 8-bit linear layer's entry points: every refusal
happens on the host, before anything touches a device."""
import ctypes

import pytest
import torch

import orthonormal_optimizer_step_gb300 as od
from orthonormal_optimizer_step_gb300 import build as odbuild

BAD, OK, UNSUPPORTED, NOSPACE = od.DION_ERR_INVALID_ARG, od.DION_OK, od.DION_ERR_UNSUPPORTED, od.DION_ERR_WORKSPACE
P = 1 << 20                                        # an address that is never read: validation fails first


@pytest.fixture(scope="module")
def lib():
    odbuild.build()
    return od.lib()


def quant(lib, **kw):
    a = dict(batch=1, rows=64, cols=256, dt=1, x=P, ldx=256, sx=0, rstd=None, weight=None, wdt=0, square=0, fmt=0,
             q=P, ldq=256, sq=0, s=P, lds=4, ss=0, qt=None, ldqt=0, sqt=0, st=None, ldst=0, sst=0, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.dion_q8_quantize(*a.values())


@pytest.mark.parametrize("kw", [
    dict(batch=-1), dict(rows=-1), dict(cols=-1), dict(dt=2), dict(fmt=2), dict(square=2), dict(wdt=5),
    dict(x=None), dict(x=P + 1), dict(ldx=255), dict(q=None), dict(s=None), dict(q=P + 8), dict(s=P + 2),
    dict(ldq=248), dict(ldq=264), dict(lds=1), dict(lds=6), dict(q=None, s=None), dict(qt=P), dict(st=P),
    dict(qt=P, st=P, ldqt=48, ldst=4), dict(qt=P, st=P, ldqt=64, ldst=0),
    dict(rstd=P), dict(weight=P), dict(rstd=P, weight=P, batch=2, sx=1 << 14, sq=1 << 14, ss=256), dict(rstd=P + 2, weight=P),
    dict(batch=2, sx=100, sq=1 << 14, ss=256), dict(batch=2, sx=1 << 14, sq=100, ss=256),
    dict(batch=2, sx=1 << 14, sq=1 << 14, ss=8), dict(batch=2, sx=1 << 14, sq=(1 << 14) + 8, ss=256),
])
def test_quantize_refuses(lib, kw):
    assert quant(lib, **kw) == BAD


def test_quantize_empty_and_too_large(lib):
    for kw in (dict(batch=0), dict(rows=0), dict(cols=0)):
        assert quant(lib, **kw) == OK
    assert quant(lib, batch=65536, sx=1 << 14, sq=1 << 14, ss=256) == UNSUPPORTED
    assert quant(lib, rows=0x7fffffff) == UNSUPPORTED


def matmul(lib, **kw):
    a = dict(m=64, n=48, k=256, a=P, lda=256, af=0, sa=P, ldsa=4, a_sq=0, b=P, ldb=256, bf=0, sb=P, ldsb=4, b_sq=0,
             c=P, ldc=48, cdt=1, status=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.dion_q8_matmul(*a.values())


@pytest.mark.parametrize("kw", [
    dict(m=-1), dict(n=-1), dict(k=-1), dict(af=2), dict(bf=-1), dict(cdt=2), dict(a_sq=2), dict(b_sq=-1),
    dict(a=None), dict(a=P + 8), dict(lda=255), dict(lda=264), dict(sa=None), dict(sa=P + 1), dict(ldsa=1),
    dict(ldsa=5), dict(b=None), dict(b=P + 4), dict(ldb=240), dict(sb=None), dict(ldsb=2), dict(c=None),
    dict(c=P + 1), dict(c=P + 2, cdt=0), dict(ldc=47), dict(status=P + 1),
])
def test_matmul_refuses(lib, kw):
    assert matmul(lib, **kw) == BAD


def test_matmul_empty(lib):
    assert matmul(lib, m=0) == OK and matmul(lib, n=0) == OK
    assert matmul(lib, lda=1 << 41) == UNSUPPORTED


def norm(lib, **kw):
    a = dict(rows=8, cols=256, dt=1, x=P, ldx=256, r=P, ldr=256, w=P, wdt=1, eps=1e-6, h=P, ldh=256, fmt=0, q=P,
             ldq=256, s=P, lds=4, rstd=P, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.dion_rms_norm_q8(*a.values())


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(cols=-1), dict(dt=3), dict(wdt=3), dict(fmt=3), dict(r=None), dict(h=None), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(x=P + 1), dict(ldx=255), dict(ldr=255),
    dict(ldh=255), dict(w=None), dict(w=P + 1), dict(w=P + 2, wdt=0), dict(q=P + 8), dict(ldq=250), dict(s=None),
    dict(lds=3), dict(rstd=P + 2),
])
def test_norm_refuses(lib, kw):
    assert norm(lib, **kw) == BAD


def test_norm_empty(lib):
    assert norm(lib, rows=0) == OK and norm(lib, cols=0) == OK


def backward(lib, **kw):
    a = dict(rows=8, cols=256, dt=1, dy=P, lddy=256, h=P, ldh=256, rstd=P, w=P, wdt=1, dh=None, lddh=0, dx=P, lddx=256,
             dw=P, ws=P, wsb=ctypes.c_size_t(1 << 30), stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.dion_rms_norm_backward(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), BAD), (dict(cols=-1), BAD), (dict(dt=2), BAD), (dict(wdt=2), BAD), (dict(dy=None), BAD),
    (dict(dy=P + 1), BAD), (dict(lddy=255), BAD), (dict(h=None), BAD), (dict(ldh=10), BAD), (dict(rstd=None), BAD),
    (dict(w=None), BAD), (dict(dh=P, lddh=255), BAD), (dict(dx=None), BAD), (dict(lddx=1), BAD), (dict(dw=None), BAD),
    (dict(dw=P + 2), BAD), (dict(ws=None), NOSPACE), (dict(ws=P + 16), NOSPACE), (dict(wsb=ctypes.c_size_t(64)), NOSPACE),
    (dict(cols=0), OK),
])
def test_backward_refuses(lib, kw, code):
    assert backward(lib, **kw) == code


def test_backward_workspace_size(lib):
    assert od.dion_rms_norm_backward_workspace_size(0, 256) == 0
    assert od.dion_rms_norm_backward_workspace_size(1, 256) == 1024
    assert lib.dion_rms_norm_backward_workspace_size(-1, 4, ctypes.byref(ctypes.c_size_t())) == BAD
    assert lib.dion_rms_norm_backward_workspace_size(4, 4, None) == BAD


def test_binding_refuses_on_cpu():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        od.dion_q8_quantize(x)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        od.dion_q8_quantize(x.half())
    with pytest.raises(TypeError, match="8-bit format"):
        od.dion_q8_quantize(x, dtype=torch.int8)
    with pytest.raises(ValueError, match="form"):
        od.dion_q8_quantize(x, form="rowwise")
    with pytest.raises(ValueError, match="rows, cols"):
        od.dion_q8_quantize(x[0])
    with pytest.raises(ValueError, match="CUDA"):
        od.dion_rms_norm_q8(x, torch.ones(256))
    with pytest.raises(ValueError, match="CUDA"):
        od.dion_rms_norm_backward(x, x, torch.ones(4), torch.ones(256))
    a = od.new_q8(4, 256, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        od.dion_q8_matmul(a, a)
    with pytest.raises(ValueError, match="expected"):
        od.dion_q8_matmul(a, od.new_q8(4, 128, device="cpu"))


def test_new_q8_layout():
    for rows, cols, square, batch in [(1, 1, False, None), (300, 1000, True, None), (5, 129, False, 3)]:
        q = od.new_q8(rows, cols, square=square, batch=batch, device="cpu")
        lead = () if batch is None else (batch,)
        assert q.data.shape == lead + (rows, cols)
        assert q.scale.shape == lead + (-(-rows // 128) if square else rows, -(-cols // 128))
        assert q.data.stride(-2) % 16 == 0 and q.scale.stride(-2) % 4 == 0
