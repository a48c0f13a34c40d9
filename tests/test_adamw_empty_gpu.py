"""AdamW plans without values."""
import math

import pytest
import torch

import orthonormal_optimizer_step_gb300 as od

pytestmark = pytest.mark.gpu


def test_plans_of_nothing_count_on_the_device():
    """A process that owns no such parameters keeps its count with the others."""
    hyper = torch.tensor([1e-3, 0.9, 0.999, 1e-8, 0.0], dtype=torch.float64, device="cuda")
    empty = [torch.empty(0, device="cuda")]
    for plan in (od.dion_adamw_plan([], [], [], []), od.dion_adamw_plan(empty, empty, *od.dion_adamw_state(empty))):
        count = torch.zeros(1, dtype=torch.int64, device="cuda")
        for t in range(1, 4):
            od.dion_adamw_step(plan, step=count, hyper=hyper)
            assert int(count) == t
        od.dion_adamw_step(plan, step=count, hyper=hyper, grad_scale=torch.tensor([math.nan], device="cuda"))
        assert int(count) == 3
        with pytest.raises(ValueError, match="hyper"):
            od.dion_adamw_step(plan, step=count, hyper=hyper.float())
        with pytest.raises(ValueError, match="step"):
            od.dion_adamw_step(plan, step=4, hyper=hyper)
        od.dion_adamw_step(plan, step=1, lr=1e-3)
