"""CPU-only checks of the 4-bit entry points: every refusal happens on the host,
before anything touches a device."""
import numpy as np
import pytest
import torch

import orthonormal_optimizer_step_gb300 as od
import q4_ref as ref
from orthonormal_optimizer_step_gb300 import build as odbuild
from orthonormal_optimizer_step_gb300 import q4

BAD, OK, UNSUPPORTED = od.DION_ERR_INVALID_ARG, od.DION_OK, od.DION_ERR_UNSUPPORTED
P = 1 << 20                                        # an address that is never read: validation fails first


@pytest.fixture(scope="module")
def lib():
    odbuild.build()
    return od.lib()


def quantize(lib, **kw):
    a = dict(rows=64, cols=200, group=128, dt=1, x=P, ldx=200, q=P, ldq=128, s=P, lds=2, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.dion_q4_quantize(*a.values())


def dequantize(lib, **kw):
    a = dict(rows=64, cols=200, group=128, q=P, ldq=128, s=P, lds=2, dt=1, x=P, ldx=200, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.dion_q4_dequantize(*a.values())


@pytest.mark.parametrize("call", [quantize, dequantize])
@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(cols=-1), dict(group=16), dict(group=0), dict(group=256), dict(dt=2), dict(x=None), dict(x=P + 1),
    dict(x=P + 2, dt=0), dict(ldx=199), dict(q=None), dict(q=P + 8), dict(ldq=120), dict(ldq=136), dict(ldq=64), dict(s=None),
    dict(s=P + 1), dict(lds=1),
])
def test_quantization_refuses(lib, call, kw):
    assert call(lib, **kw) == BAD


@pytest.mark.parametrize("call", [quantize, dequantize])
def test_quantization_empty_and_too_large(lib, call):
    assert call(lib, rows=0) == OK and call(lib, cols=0) == OK
    assert call(lib, rows=0x7fffffff) == UNSUPPORTED


def matmul(lib, **kw):
    a = dict(m=2, n=64, k=200, xt=1, x=P, ldx=200, sx=None, ldsx=0, group=128, q=P, ldq=128, s=P, lds=2, ydt=1, y=P, ldy=64,
             stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.dion_q4_matmul(*a.values())


@pytest.mark.parametrize("kw", [
    dict(m=-1), dict(n=-1), dict(k=-1), dict(xt=4), dict(xt=-1), dict(group=48), dict(ydt=2), dict(x=None), dict(x=P + 1),
    dict(x=P + 2, xt=0), dict(ldx=199), dict(q=P + 4), dict(ldq=100), dict(s=None), dict(lds=1), dict(y=None), dict(y=P + 1),
    dict(y=P + 2, ydt=0), dict(ldy=63),
    dict(xt=2, ldx=208, sx=None, ldsx=4), dict(xt=2, ldx=208, sx=P + 2, ldsx=4), dict(xt=2, ldx=208, sx=P, ldsx=2),
    dict(xt=3, ldx=200, sx=P, ldsx=4), dict(xt=3, x=P + 8, ldx=208, sx=P, ldsx=4),
])
def test_matmul_refuses(lib, kw):
    assert matmul(lib, **kw) == BAD


def test_matmul_empty_and_too_large(lib):
    assert matmul(lib, m=0) == OK and matmul(lib, n=0) == OK
    assert matmul(lib, m=65536) == UNSUPPORTED
    assert matmul(lib, k=131073, ldx=131073, ldq=64 * 1025, lds=1025) == UNSUPPORTED
    assert matmul(lib, n=0x7fffffff, ldy=0x7fffffff) == UNSUPPORTED


# ------------------------------------------------------------------- binding
def test_new_matrices_are_aligned():
    w = od.new_q4(5, 1000, group=64, device="cpu")
    assert w.data.shape == (5, 512) and w.scale.shape == (5, 16) and w[2:] == (1000, 64)
    assert od.new_q4(5, 300, group=32, device="cpu").scale.stride() == (16, 1)
    with pytest.raises(ValueError, match="group"):
        od.new_q4(5, 300, group=48, device="cpu")


def test_matrices_that_do_not_fit_are_refused():
    w = od.new_q4(4, 300, group=64, device="cpu")
    assert q4._q4(w, "w")[:3] == (4, 300, 64)
    for bad, error in ((w._replace(group=100), ValueError), (w._replace(cols=400), ValueError), (w._replace(cols=-1), ValueError),
                       (w._replace(scale=w.scale.float()), TypeError), (w._replace(data=w.data.view(torch.int8)), TypeError),
                       (w._replace(data=w.data[:3]), ValueError), (w._replace(scale=w.scale[:, :4]), ValueError),
                       (w._replace(data=torch.empty(4 * 192 + 8, dtype=torch.uint8)[8:].view(4, 192)), ValueError),
                       (w._replace(data=torch.empty(4, 200, dtype=torch.uint8)[:, :192]), ValueError),
                       (w._replace(data=w.data[0]), ValueError)):
        with pytest.raises(error):
            q4._q4(bad, "w")


def test_tensors_of_the_cpu_are_refused():
    w = od.new_q4(4, 300, device="cpu")
    for call in (lambda: od.dion_q4_quantize(torch.zeros(4, 300)), lambda: od.dion_q4_dequantize(w),
                 lambda: od.dion_q4_matmul(torch.zeros(1, 300), w)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_reference_layout_is_a_permutation():
    q = torch.from_numpy(np.random.RandomState(0).randint(-8, 8, (3, 300)).astype(np.int8))
    assert sorted(ref.column_of_nibble(300)) == list(range(384))
    assert torch.equal(ref.unpack(ref.pack(q), 300)[:, :300], q.to(torch.int16))
    # the first word: columns 0 2 4 6 1 3 5 7, the second's first column 32, the fifth's 8
    assert ref.column_of_nibble(128)[:9] == [0, 2, 4, 6, 1, 3, 5, 7, 32] and ref.column_of_nibble(128)[32] == 8
