"""4-bit products of rows and weights at the ends of float32's range."""
import pytest
import torch

import orthonormal_optimizer_step_gb300 as od
from test_q4_gpu import matrix, values

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("kind", [F32, BF16])
@pytest.mark.parametrize("std,weight", [(1.0, 1.0), (1e-29, 1.0), (1e-33, 1.0), (1e-36, 1e10), (1e-38, 1e10), (1e-41, 1e10), (1e30, 1e-10)])
@pytest.mark.parametrize("m", [1, 5, 20])
def test_rows_of_small_and_large_values(kind, std, weight, m):
    """Weights that are a diagonal: each product by itself, so that what x loses shows.

    float32: 2^-24 of a value and 2^-39 of the largest of its 128 columns; bfloat16: the
    latter alone; each result has two roundings more.  (Of 1e-41 bfloat16 has nothing: its
    least number is 9.2e-41, so all values round to zero.)"""
    k = 300
    w = od.dion_q4_quantize(torch.eye(k, device="cuda") * 7 * weight, group=32)
    x = (matrix(m, k, F32, 1, 1.0).double() * std).to(kind)
    xv, scale = x.double(), values(w).diagonal()
    want = xv * scale
    largest = torch.nn.functional.pad(xv, (0, -k % 128)).view(m, -1, 128).abs().amax(-1).repeat_interleave(128, 1)[:, :k]
    slack = (3 if kind is F32 else 2) * 2.0 ** -24 * want.abs() + 2.0 ** -39 * largest * scale
    y = od.dion_q4_matmul(x, w, out_dtype=F32)
    assert torch.all((y.double() - want).abs() <= slack) and bool(y.any()) == bool(want.any())


@pytest.mark.parametrize("kind", [F32, BF16])
@pytest.mark.parametrize("std,weight", [(1e-33, 1.0), (1e-38, 1e10), (1e30, 1e-10)])
@pytest.mark.parametrize("m,n,k", [(1, 64, 1000), (5, 200, 4096), (20, 33, 520)])
def test_sums_of_small_and_large_values(kind, std, weight, m, n, k):
    """The chain of sums (16 terms each, truncated: 2^-23) and what x loses."""
    w = od.dion_q4_quantize(matrix(n, k, F32, std=weight))
    x = (matrix(m, k, F32, 1, 1.0).double() * std).to(kind)
    xv, wv = x.double(), values(w)
    chain = k / 16 + k / w.group + k / 128 + 16
    size, far = xv.abs() @ wv.abs().t(), 2.0 ** -39 * xv.abs().amax(1, keepdim=True) * wv.abs().sum(1)
    y = od.dion_q4_matmul(x, w, out_dtype=F32)
    assert torch.all((y.double() - xv @ wv.t()).abs() <= (chain * 2.0 ** -23 + 2.0 ** -23) * size + far)
