"""8-bit first moments over many steps: they follow their gradients, and come to rest with them."""
import math

import pytest
import torch

import adamw_ref as ref
import orthonormal_optimizer_step_gb300 as od

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def low_dither(n, seed, t, index):
    """The first moment's dither in (0, 1): the hash's lower 12 bits, and a half."""
    key = ref.mix(ref.mix((seed * 0x632BE5AB + t) & 0xFFFFFFFF) ^ ref.np.uint64(index))
    h = ref.mix(ref.np.arange(n, dtype=ref.np.uint64) ^ key)
    return torch.from_numpy(((h & ref.np.uint64(0xFFF)).astype(ref.np.float64) + 0.5) / 4096)


def check_dithered(state, want, terms, u, where=None):
    """A State8 of first moments rounded by their dither, within what float32 leaves open.

    As in check8: 2^-21 of a value, 2^-22 of its terms, and 2^-29 are granted to what is rounded."""
    n = want.numel()
    s = state.scale.double().repeat_interleave(256)[:n]
    y, got = want / s, state.data.flatten().double()
    step, slack = ref.spacing(y.abs()), 2.0 ** -21 * y.abs() + 2.0 ** -29 + 2.0 ** -22 * terms / s
    low = (torch.floor((y.abs() - slack).clamp(min=0) / step + u) * step).clamp(max=448)
    high = (torch.floor((y.abs() + slack) / step + u) * step).clamp(max=448)
    edge = (torch.log2(y.abs().clamp(min=1e-300)) - torch.round(torch.log2(y.abs().clamp(min=1e-300)))).abs() < 2.0 ** -18
    ok = ((got.abs() >= low) & (got.abs() <= high)) | (edge & ((got.abs() - y.abs()).abs() <= step))
    ok &= (got == 0) | (torch.sign(got) == torch.sign(y))
    assert torch.all(ok if where is None else ok[where])


def states(n, seed):
    """8-bit states of Gaussian codes, as after some steps."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    first = (torch.randn(n, generator=gen, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    second = (torch.randn(n, generator=gen, device="cuda") * 100).abs().clamp(max=448).to(torch.float8_e4m3fn)
    scales = [torch.rand(-(-n // 256), generator=gen, device="cuda") * 1e-5 + 1e-6 for _ in range(2)]
    return od.State8(first, scales[0]), od.State8(second, scales[1]), gen


@pytest.mark.parametrize("beta1", [0.0, 0.9, 0.95, 0.99])
@pytest.mark.parametrize("p", [F32, BF16])
@pytest.mark.parametrize("n", [1, 255, 5000, 3_000_003])
def test_codes_follow_from_the_dither(beta1, p, n):
    """Every value with beta1 above 29/32; below, values under 2^-6 whose gradient's part is at most 2^-9 (of the scale)."""
    first, second, gen = states(n, 3)
    g = torch.randn(n, generator=gen, device="cuda") * 1e-3
    small = torch.arange(n, device="cuda") % 7 == 3
    first.data.copy_(torch.where(small, first.data.float() / 4096, first.data.float()).to(torch.float8_e4m3fn))
    g[small] *= 2.0 ** -13
    m = ref.values(first, n)
    params = torch.zeros(n, device="cuda", dtype=p)
    plan = od.dion_adamw_plan([params], [g], [first], [second])
    od.dion_adamw_step(plan, step=5, lr=1e-3, betas=(beta1, 0.999), seed=11)
    part = (1 - beta1) * g.double()
    want, terms = beta1 * m + part, beta1 * m.abs() + part.abs()
    u = low_dither(n, 11, 5, 0).cuda()
    if 1 - beta1 < 3 / 32:
        check_dithered(first, want, terms, u)
        return
    s = first.scale.double().repeat_interleave(256)[:n]
    near = (want / s).abs() < 2.0 ** -6 - 2.0 ** -9         # (what nearest rounding takes to 2^-6 is left as it is)
    inside = near & (part.abs() / s <= 2.0 ** -9 * (1 - 2.0 ** -12))
    assert n < 5000 or int(inside.sum()) > n // 200
    check_dithered(first, want, terms, u, inside)
    outside = ((want / s).abs() > 2.0 ** -6) | (part.abs() / s > 2.0 ** -9 * (1 + 2.0 ** -12))
    y, got = (want / s)[outside], first.data.double()[outside]
    slack = 2.0 ** -21 * y.abs() + 2.0 ** -29 + (2.0 ** -22 * terms / s)[outside]
    assert torch.all((got - y).abs() <= ref.spacing(y.abs()) / 2 + slack)


@pytest.mark.parametrize("betas,rest", [((0.9, 0.95), 500), ((0.9, 0.999), 500), ((0.95, 0.99), 800), ((0.99, 0.999), 4000)])
@pytest.mark.parametrize("p", [F32, BF16])
def test_parameters_without_gradients_come_to_rest(betas, rest, p):
    """One value of eight has no gradient after 200 steps: its first moment reaches zero, and the parameter stays.

    A dithered moment is a whole number of least codes whose mean falls by beta1 a step, so
    512 values are all zero after k steps but for a chance of 512 c beta1^k, c being where
    the dither takes over (the blocks' scales, which the others' gradients move, double it).
    beta1 = 0.9: c is 7, after the nearest rounding's at most 200 steps (0.9 * 17 / 16 of a
    value each at most); 300 more leave 1e-9.  The others: c is 448 * 512, and the chance
    1e-9 or less."""
    n = 4096
    params, grad = torch.zeros(n, device="cuda", dtype=p), torch.empty(n, device="cuda")
    first, second = od.dion_adamw_state([params], bits=8)
    plan = od.dion_adamw_plan([params], [grad], first, second)
    gen = torch.Generator(device="cuda").manual_seed(2)
    idle = torch.arange(n, device="cuda") % 8 == 3
    for t in range(1, 200 + rest + 51):
        if t == 200 + rest + 1:
            assert not first[0].data[idle].float().any()
            held = params.clone()
        grad.copy_(torch.randn(n, generator=gen, device="cuda") * 1e-3)
        if t > 200:
            grad[idle] = 0
        od.dion_adamw_step(plan, step=t, lr=1e-3, betas=betas)
    assert torch.equal(params[idle], held[idle]) and not torch.equal(params, held)


def test_narrow_rows_that_are_no_longer_used_stay():
    """An embedding of width 64, four rows a block, one of four unused from step 200 on: decay alone moves it."""
    rows, width = 64, 64
    table = torch.zeros(rows, width, device="cuda")
    grad = torch.empty_like(table)
    first, second = od.dion_adamw_state([table], bits=8)
    plan = od.dion_adamw_plan([table], [grad], first, second)
    gen = torch.Generator(device="cuda").manual_seed(5)
    for t in range(1, 3001):
        if t == 701:
            held = table[1::4].double()
        grad.copy_(torch.randn(rows, width, generator=gen, device="cuda") * 1e-3)
        if t > 200:
            grad[1::4] = 0
        od.dion_adamw_step(plan, step=t, lr=1e-3, betas=(0.9, 0.95), weight_decay=0.1)
    # 2300 steps of decay by 1e-4, each rounded to float32 (the step and lr * weight_decay too: 4 half steps a step of p)
    want = held * (1 - 1e-4) ** 2300
    assert torch.all((table[1::4].double() - want).abs() <= 2300 * 4 * 2.0 ** -24 * held.abs())


@pytest.mark.parametrize("beta1,start,g,steps", [(0.9, 10, -3.0, 400), (0.99, 128 * 512, 40 * 512.0, 200)])
def test_moments_follow_a_gradient_that_changes_them_by_less_than_a_step(beta1, start, g, steps):
    """Means of dithered moments are the formula's: sums of the step's changes, each without bias.

    In least codes, 2^-9 of a scale that one value of each block holds.  A step's variance is
    at most a quarter of the distance's square (1 below 16; 16 * 512 below 256 * 512), all of
    them together that divided by 1 - beta1^2, and the mean of 4080 values has 1/4080 of it:
    six deviations.  The dither's 12 bits are off by 2^-13 of a distance a step, float32 by
    less."""
    n = 4096
    grad = torch.full((n,), g * 2.0 ** -9 / 448 * 1e-3, device="cuda")
    grad[::256] = 1e-3
    params = [torch.zeros(n, device="cuda")]
    first, second = od.dion_adamw_state(params, bits=8)
    for s, code in ((first[0], start * 2.0 ** -9), (second[0], 448.0)):
        s.scale.fill_(1e-3 / 448)
        s.data.copy_(torch.full((n,), code, device="cuda").to(torch.float8_e4m3fn))
        s.data.view(torch.uint8)[::256] = 126                # 448
    plan = od.dion_adamw_plan(params, [grad], first, second)
    for t in range(1, steps + 1):
        od.dion_adamw_step(plan, step=t, lr=0.0, betas=(beta1, 0.999))
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[::256] = False
    got = float((ref.values(first[0], n)[keep] / (1e-3 / 448) * 512).mean())
    want = g + (start - g) * beta1 ** steps
    distance = 1.0 if start < 16 else 16 * 512.0
    slack = 6 * distance / 2 / math.sqrt((1 - beta1 ** 2) * 4080) + (2.0 ** -13 + 2.0 ** -20) * distance / (1 - beta1)
    assert abs(got - want) <= slack


@pytest.mark.parametrize("beta1", [0.9, 0.99])
def test_what_is_not_finite_has_its_own_code(beta1):
    n = 512
    g = torch.randn(n, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") * 1e-3
    g[3], g[300], g[400] = math.inf, -math.inf, math.nan
    params = [torch.zeros(n, device="cuda")]
    first, second = od.dion_adamw_state(params, bits=8)
    od.dion_adamw_step(od.dion_adamw_plan(params, [g], first, second), step=1, lr=1e-3, betas=(beta1, 0.999))
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[[3, 300, 400]] = True
    assert torch.equal(torch.isnan(first[0].data.float()), bad) and torch.isfinite(first[0].scale).all()


@pytest.mark.parametrize("beta1", [0.9, 0.95])
def test_mixed_lists_and_device_numbers_have_the_same_bits(beta1):
    """8-bit states among float32 ones, and with hyperparameters on the device, against a list of their own with numbers."""
    n, other = 2_000_003, 70_001
    hyper = torch.tensor([1e-3, beta1, 0.999, 1e-8, 0.1], dtype=torch.float64, device="cuda")
    runs = []
    for mixed, device in ((False, False), (True, False), (False, True), (True, True)):
        first, second, gen = states(n, 3)
        g = torch.randn(n, generator=gen, device="cuda") * 1e-3
        g[::3] *= 1e-5
        p = torch.randn(n, generator=gen, device="cuda")
        lists = [p], [g], [first], [second]
        if mixed:
            more = [torch.randn(other, generator=gen, device="cuda") for _ in range(3)]
            for to, x in zip(lists, (*more, more[0].square())):
                to.append(x)
        plan = od.dion_adamw_plan(*lists)
        if device:
            od.dion_adamw_step(plan, step=torch.full((1,), 6, dtype=torch.int64, device="cuda"), hyper=hyper, seed=4)
        else:
            od.dion_adamw_step(plan, step=7, lr=1e-3, betas=(beta1, 0.999), weight_decay=0.1, seed=4)
        runs.append([p, first.data.view(torch.uint8), first.scale, second.data.view(torch.uint8), second.scale])
    for run in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], run))
