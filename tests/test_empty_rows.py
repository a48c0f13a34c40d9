"""Rows without columns, with leading dimensions."""
import pytest
import torch

import orthonormal_optimizer_step_gb300 as od
from orthonormal_optimizer_step_gb300 import q8


@pytest.mark.parametrize("shape", [(2, 3, 0), (2, 0, 5), (0, 3, 0), (4, 0), (1, 1, 0)])
def test_are_a_matrix_of_rows(shape):
    t, ld = q8._matrix(torch.empty(shape), "x")
    rows = 1
    for n in shape[:-1]:
        rows *= n
    assert t.shape == (rows, shape[-1]) and ld >= shape[-1]


@pytest.mark.gpu
def test_products_of_nothing_are_zeros():
    none = od.dion_q4_quantize(torch.empty(48, 0, device="cuda"))
    y = od.dion_q4_matmul(torch.empty(2, 3, 0, device="cuda"), none)
    assert y.shape == (2, 3, 48) and not y.any()
