"""Weight decay of AdamW: what float32 has no room for beside one, and parameters that are not finite."""
import math

import pytest
import torch

import adamw_ref as ref
import orthonormal_optimizer_step_gb300 as od
from test_adamw_gpu import make

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("decay", [1e-7, 2e-8, 3e-6])
def test_small_decays_count(bits, decay):
    """lr * weight_decay below float32's 2^-24 beside one: each parameter is its value in 64 bits, rounded.

    A result below 2 is rounded by 2^-24 at most (from 2 on by 2^-23); the update and the
    decay, before that, are right to 20 half steps of their own.  (Decays of 1e-7, 2e-8 and
    3e-6 as multiples of 2^-24 are off by 1.9e-8, 2e-8 and 2e-8 of a parameter, a third of
    2^-24 and more.)"""
    n, lr, t = 1 << 20, 1e-6, 7
    _, (g,), (first,), (second,), _ = make([n], bits=bits)
    p = 1 + torch.rand(n, generator=torch.Generator(device="cuda").manual_seed(8), device="cuda")
    m, v = (ref.values(first, n), ref.values(second, n).square()) if bits == 8 else (first.double(), second.double())
    want, _, _, size = ref.step(p, g, m, v, t, lr=lr, weight_decay=decay / lr)
    before = p.double()
    od.dion_adamw_step(od.dion_adamw_plan([p], [g], [first], [second]), step=t, lr=lr, weight_decay=decay / lr)
    half = torch.where(want < 2, 2.0 ** -24, 2.0 ** -23)
    assert torch.all((p.double() - want).abs() <= half + 20 * 2.0 ** -24 * (size + decay * before))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p", [F32, BF16])
@pytest.mark.parametrize("decay", [0.0, 0.1])
def test_infinite_parameters_stay(bits, p, decay):
    """A parameter that masks (minus infinity, without a gradient) is what it was; its neighbours step as without it."""
    n = 3000
    gen = torch.Generator(device="cuda").manual_seed(9)
    plain = torch.randn(n, generator=gen, device="cuda").to(p)
    params, grad = plain.clone(), torch.randn(n, generator=gen, device="cuda") * 1e-3
    bad = torch.arange(n, device="cuda") % 97 == 5
    params[bad] = torch.where(torch.arange(int(bad.sum()), device="cuda") % 2 == 0, math.inf, -math.inf).to(p)
    held = params[bad].clone()
    for x in (params, plain):
        first, second = od.dion_adamw_state([x], bits=bits)
        od.dion_adamw_step(od.dion_adamw_plan([x], [grad], first, second), step=1, lr=1e-2, weight_decay=decay)
    assert torch.equal(params[bad], held) and torch.equal(params[~bad], plain[~bad])
