"""Forms of the norm, its gradient and the quantization that need particular
sizes, types or values to be reached, against 64 bits with the tolerances of
test_q8_gpu, and the norm's stored sum bit for bit."""
import pytest
import torch

import orthonormal_optimizer_step_gb300 as od
from test_q8_gpu import BF16, E4M3, E5M2, F32, NORM_SIZES, STREAM_SIZES, randn

pytestmark = pytest.mark.gpu


def launched(call):
    """The call's result and the names of the kernels it launched."""
    with od.profile() as p:
        got = call()
    torch.cuda.synchronize()
    return got, set(p.read())


# ------------------------------------------------------ the norm's stored sum
def special_sums(x, r):
    """Puts values into x and r whose sum is not finite, zero, or rounds at a tie."""
    inf, nan = float("inf"), float("nan")
    for i, (a, b) in enumerate([(inf, 1.0), (1.0, -inf), (inf, -inf), (nan, 2.0), (3.3e38, 3.3e38), (-0.0, 0.0),
                                (-0.0, -0.0), (1.0, 2.0 ** -8), (1.0, 3 * 2.0 ** -8), (1e-40, -1e-40), (256.0, 1.0)]):
        n = x.numel()
        at = (i * 7919) % n
        x.view(-1)[at], r.view(-1)[at] = a, b


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("special", [False, True])
@pytest.mark.parametrize("rows,cols", NORM_SIZES + STREAM_SIZES)
def test_norm_stores_the_rounded_sum(rows, cols, special, dtype):
    x, r, w = randn(rows, cols, dtype=dtype), randn(rows, cols, dtype=dtype, seed=2, std=3.0), randn(cols, seed=1)
    if special:
        special_sums(x, r)
    want = (x.float() + r.float()).to(dtype)
    _, h, _ = od.dion_rms_norm_q8(x, w, residual=r)
    torch.testing.assert_close(h, want, rtol=0, atol=0, equal_nan=True)
    assert torch.equal(torch.signbit(h)[~torch.isnan(h)], torch.signbit(want)[~torch.isnan(want)])
