"""The scales up to which 4-bit products cannot overflow between their steps."""
import pytest
import torch

import orthonormal_optimizer_step_gb300 as od

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("group", [32, 128])
def test_scales_up_to_the_stated_bound(kind, group):
    """Weights of 7 * 2^101 and all activations at their largest: no sum between overflows, and the product is finite."""
    k = 1024
    w = od.dion_q4_quantize(torch.full((48, k), 7 * 2.0 ** 101, device="cuda"), group=group)
    assert float(w.scale[0, 0]) == 2.0 ** 101
    if kind == "e4m3":
        x = od.dion_q8_quantize(torch.full((3, k), 1.75 * 2.0 ** -60, device="cuda"))[0]
    else:
        x = torch.full((3, k), (2 - 2.0 ** -7) * 2.0 ** -60, device="cuda").to(F32 if kind == "f32" else BF16)
    want = 1024 * 7 * 2.0 ** 41 * (1.75 if kind == "e4m3" else 2 - 2.0 ** -7)
    y = od.dion_q4_matmul(x, w, out_dtype=F32)
    assert torch.all((y.double() - want).abs() <= (k / 16 + k / group + k / 128 + 17) * 2.0 ** -23 * want)
