"""The norm of gradients whose squares leave float32's normal numbers."""
import pytest
import torch

import orthonormal_optimizer_step_gb300 as od

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1000, 3_000_001])
def test_norm_of_small_gradients(n):
    """Squares around 1e-40 are subnormal: each is off by half of 2^-149 at most, their sums are exact."""
    g = torch.randn(n, generator=torch.Generator(device="cuda").manual_seed(7), device="cuda") * 1e-20
    want = float(g.double().square().sum())
    norm, factor = od.dion_grad_norm(od.dion_grad_list([g]), max_norm=1.0).tolist()
    assert abs(norm ** 2 - want) <= n * 2.0 ** -150 + 40 * 2.0 ** -24 * want and factor == 1.0
    # below 2^-75 a square is nothing
    assert od.dion_grad_norm(od.dion_grad_list([torch.full((n,), 2.0 ** -76, device="cuda")])).tolist() == [0.0, 1.0]
