"""AdamW with epsilons at the end of float32's range."""
import pytest
import torch

import orthonormal_optimizer_step_gb300 as od

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-38, 1e-40, 1e-50])
@pytest.mark.parametrize("device", [False, True])
def test_epsilons_below_the_least_normal_number(bits, eps, device):
    """Nothing divided by an epsilon is nothing, however small the epsilon."""
    p = [torch.ones(300, device="cuda")]
    first, second = od.dion_adamw_state(p, bits=bits)
    plan = od.dion_adamw_plan(p, [torch.zeros(300, device="cuda")], first, second)
    if device:
        hyper = torch.tensor([1e-3, 0.9, 0.999, eps, 0.0], dtype=torch.float64, device="cuda")
        od.dion_adamw_step(plan, step=torch.zeros(1, dtype=torch.int64, device="cuda"), hyper=hyper)
    else:
        od.dion_adamw_step(plan, step=1, lr=1e-3, eps=eps)
    assert torch.all(p[0] == 1)
