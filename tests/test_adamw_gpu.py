"""AdamW over many tensors and the gradients' norm against float64."""
import math

import pytest
import torch

import adamw_ref as ref
import orthonormal_optimizer_step_gb300 as od

pytestmark = pytest.mark.gpu

EPS32, HALF = 2.0 ** -24, {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F32, BF16 = torch.float32, torch.bfloat16


def make(sizes, p=F32, g=F32, bits=32, seed=0, offset=0, copies=False):
    """Parameters, gradients and states that have seen some steps; `offset`: elements between a tensor and its allocation."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def new(n, std, dtype):
        t = (torch.randn(n + offset, generator=gen, device="cuda") * std).to(dtype)
        return t[offset:]

    params, grads = [new(n, 0.02, p) for n in sizes], [new(n, 1e-3, g) for n in sizes]
    if bits == 32:
        first, second = [new(n, 3e-4, F32) for n in sizes], [new(n, 1e-3, F32).square_() for n in sizes]
    else:
        first, second = [], []
        for n in sizes:
            for to in (first, second):
                q = new(n, 100.0, F32).abs().clamp(max=448).to(torch.float8_e4m3fn)
                if to is first:
                    q = (q.float() * torch.where(torch.rand(n, generator=gen, device="cuda") < 0.5, -1.0, 1.0)).to(q.dtype)
                    # (a conversion's result starts its allocation: put it where the others are)
                held = torch.empty(n + offset, dtype=torch.uint8, device="cuda").view(q.dtype)[offset:]
                held.view(torch.uint8).copy_(q.view(torch.uint8))
                blocks = -(-n // 256)
                to.append(od.State8(held, torch.rand(blocks, generator=gen, device="cuda") * 1e-5 + 1e-6))
    return params, grads, first, second, [torch.empty(n + offset, dtype=BF16, device="cuda")[offset:] for n in sizes] if copies else None


def copy_of(x):
    return od.State8(x.data.clone(), x.scale.clone()) if isinstance(x, od.State8) else x.clone()


def check(parts, before, t, seed=0, scale=1.0, index=None, lr_factors=None, decay_factors=None, lr=1e-3, wd=0.0, **kw):
    """Each result of a step within the roundings of its formula."""
    params, grads, first, second, copies = parts
    p0, m0, v0 = before
    for i, p in enumerate(params):
        n = p.numel()
        eight = isinstance(m0[i], od.State8)
        m, v = (ref.values(m0[i], n), ref.values(v0[i], n) ** 2) if eight else (m0[i].double(), v0[i].double())
        f = lr_factors[i] if lr_factors else 1.0
        want, m1, v1, size = ref.step(p0[i], grads[i], m, v, t, lr=lr * f, scale=scale,
                                      weight_decay=wd * (decay_factors[i] if decay_factors else 1.0), **kw)
        # the update: its constants, m (3 roundings of its terms), the root and the quotient (2 units each), 4 products
        slack = 20 * EPS32 * size + 3 * EPS32 * want.abs() + 2 * EPS32 * p0[i].double().abs()
        assert torch.all((p.double() - want).abs() <= slack + HALF[p.dtype] * want.abs() * (p.dtype is BF16)), i
        if copies:
            assert torch.equal(copies[i], p.to(BF16))
        terms = 0.9 * m.abs() + 0.1 * (grads[i].double() * scale).abs()
        if eight:
            ref.check8(first[i], m1, terms=terms)
            ref.check8(second[i], v1.sqrt(), ref.dither(n, seed, t, i if index is None else index[i]))
        else:
            assert torch.all((first[i].double() - m1).abs() <= 4 * EPS32 * terms)
            assert torch.all((second[i].double() - v1).abs() <= 6 * EPS32 * v1)


SIZES = [1, 7, 8, 255, 256, 257, 0, 2047, 2048, 2049, 4096, 100003]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p", [F32, BF16])
@pytest.mark.parametrize("g", [F32, BF16])
@pytest.mark.parametrize("offset", [0, 3, 8])
def test_step(bits, p, g, offset):
    parts = make(SIZES, p, g, bits, offset=offset, copies=p is F32 and offset != 8)
    before = [copy_of(x) for x in parts[0]], [copy_of(x) for x in parts[2]], [copy_of(x) for x in parts[3]]
    plan = od.dion_adamw_plan(*parts[:4], copies=parts[4])
    od.dion_adamw_step(plan, step=7, lr=1e-3, weight_decay=0.1, seed=5)
    check(parts, before, 7, seed=5, wd=0.1)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p,g", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
def test_several_chunks_a_cta(bits, p, g):
    """More chunks of 2048 than CTAs of a launch, so that each takes several through its copies in flight."""
    parts = make([9_000_003], p, g, bits, copies=p is F32)
    before = [copy_of(x) for x in parts[0]], [copy_of(x) for x in parts[2]], [copy_of(x) for x in parts[3]]
    od.dion_adamw_step(od.dion_adamw_plan(*parts[:4], copies=parts[4]), step=3, lr=1e-3)
    check(parts, before, 3)


@pytest.mark.parametrize("bits", [32, 8])
def test_lists_of_all_types_have_the_same_bits_as_single_tensors(bits):
    """A CTA's warps go from tensor to tensor by themselves: what one copies for the next tensor must not meet what
    another still reads of the last one, whatever the types."""
    types = [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)] * 3
    kinds = [make([2_000_000 + 2048 * i], p, g, bits, seed=i) for i, (p, g) in enumerate(types)]
    joined = [[copy_of(t) for k in kinds for t in k[i]] for i in range(4)]
    od.dion_adamw_step(od.dion_adamw_plan(*joined), step=3, lr=1e-3)
    for i in range(len(kinds)):
        # (the dither goes by the place in the list)
        empty = [[x[:0] if not isinstance(x, od.State8) else od.State8(x.data[:0], x.scale[:0]) for x in kinds[i][j]] * i for j in range(4)]
        alone = [empty[j] + kinds[i][j] for j in range(4)]
        od.dion_adamw_step(od.dion_adamw_plan(*alone), step=3, lr=1e-3)
        for j in (0, 2, 3):
            a, b = joined[j][i], alone[j][i]
            for s, t in zip(a, b) if isinstance(a, od.State8) else [(a, b)]:
                assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))


@pytest.mark.parametrize("offset", [0, 4, 12])
def test_lists_of_both_kinds_of_states(offset):
    """Float32 and 8-bit states in turn; 4 and 12 float32 values are 16-byte boundaries but not 32-byte ones."""
    kinds = [make([n], p, g, bits, seed=n, offset=offset) for n, p, g, bits in
             [(4_000_000, BF16, BF16, 8), (70_001, F32, F32, 32), (6_000_001, F32, BF16, 32), (2048, BF16, F32, 8), (2_000_000, F32, F32, 8)]]
    parts = [[t for k in kinds for t in k[i]] for i in range(4)] + [None]
    before = [copy_of(x) for x in parts[0]], [copy_of(x) for x in parts[2]], [copy_of(x) for x in parts[3]]
    od.dion_adamw_step(od.dion_adamw_plan(*parts[:4]), step=3, lr=1e-3)
    check(parts, before, 3)


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_in_a_row_from_nothing(bits):
    """From zeroed states, with gradients that are zero in places (rows of an embedding that no token used)."""
    parts = make([3000, 513], BF16, BF16, bits)
    params, grads = parts[:2]
    first, second = od.dion_adamw_state(params, bits=bits)
    plan = od.dion_adamw_plan(params, grads, first, second)
    gen = torch.Generator(device="cuda").manual_seed(4)
    for t in range(1, 5):
        for g in grads:
            g.copy_(torch.randn(g.shape, generator=gen, device="cuda") * 1e-3)
            g[100:400] = 0
        before = [copy_of(x) for x in params], [copy_of(x) for x in first], [copy_of(x) for x in second]
        od.dion_adamw_step(plan, step=t, lr=1e-3, weight_decay=0.0)
        check((params, grads, first, second, None), before, t)
        assert torch.equal(params[0][100:400], before[0][0][100:400])       # 0 / (0 + eps): as it was


def test_factors_and_many_tensors():
    """More tensors than one launch takes, types and states mixed, each with factors of its own."""
    lists = [make([37 + i % 11 for i in range(150)], p, g, bits, seed=i) for i, (p, g, bits) in enumerate(
        [(F32, F32, 32), (BF16, F32, 8), (F32, BF16, 8), (BF16, BF16, 32), (F32, BF16, 32)])]
    params, grads, first, second = (sum((x[k] for x in lists), []) for k in range(4))
    lrs, decays = [0.5 + i % 3 for i in range(750)], [float(i % 2) for i in range(750)]
    before = [copy_of(x) for x in params], [copy_of(x) for x in first], [copy_of(x) for x in second]
    plan = od.dion_adamw_plan(params, grads, first, second, lr_factors=lrs, decay_factors=decays)
    od.dion_adamw_step(plan, step=2, lr=1e-3, weight_decay=0.1, betas=(0.9, 0.999), seed=9)
    check((params, grads, first, second, None), before, 2, seed=9, lr_factors=lrs, decay_factors=decays, wd=0.1)


def test_a_slice_of_a_block_is_its_own():
    """What lies behind a tensor's last value in its allocation stays as it was."""
    p, g = torch.ones(512, device="cuda", dtype=BF16), torch.ones(300, device="cuda", dtype=BF16)
    data = [torch.full((512,), 9.0, device="cuda").to(torch.float8_e4m3fn) for _ in range(2)]
    scale = [torch.full((4,), 1.0, device="cuda") for _ in range(2)]
    plan = od.dion_adamw_plan([p[:300]], [g], [od.State8(data[0][:300], scale[0][:2])], [od.State8(data[1][:300], scale[1][:2])])
    od.dion_adamw_step(plan, step=1, lr=0.1)
    assert torch.all(p[300:] == 1) and not torch.any(p[:300] == 1)
    for d, s in zip(data, scale):
        assert torch.all(d.float()[300:] == 9) and torch.all(s[2:] == 1)


@pytest.mark.parametrize("bits", [32, 8])
def test_infinities_and_nan_stay_where_they_are(bits):
    parts = make([1000], F32, F32, bits)
    params, grads, first, second, _ = parts
    bad = [3, 299, 700]
    for i, v in zip(bad, (math.inf, -math.inf, math.nan)):
        grads[0][i] = v
    before = [copy_of(x) for x in params], [copy_of(x) for x in first], [copy_of(x) for x in second]
    od.dion_adamw_step(od.dion_adamw_plan(*parts[:4]), step=3, lr=1e-3)
    ok = torch.ones(1000, dtype=torch.bool, device="cuda")
    ok[bad] = False
    assert torch.all(torch.isfinite(params[0][ok])) and torch.all(torch.isnan(params[0][bad]))
    if bits == 8:
        n = 1000
        m, v = ref.values(before[1][0], n), ref.values(before[2][0], n) ** 2
        _, m1, v1, _ = ref.step(before[0][0], grads[0], m, v, 3)
        ref.check8(first[0], m1, terms=0.9 * m.abs() + 0.1 * grads[0].double().abs())
        ref.check8(second[0], v1.sqrt(), ref.dither(n, 0, 3, 0))
    else:
        assert torch.all(torch.isfinite(first[0][ok])) and torch.all(torch.isfinite(second[0][ok]))


def test_no_root_above_zero_becomes_zero():
    """Values of very different sizes in a block: the smallest keep the least code, so no update is divided by eps alone."""
    g = torch.logspace(-18, 0, 256, device="cuda")
    p = [torch.zeros(256, device="cuda")]
    first, second = od.dion_adamw_state(p, bits=8)
    od.dion_adamw_step(od.dion_adamw_plan(p, [g], first, second), step=1, lr=1e-3)
    assert torch.all(second[0].data.float() >= 2.0 ** -9)
    z = [torch.zeros(256, device="cuda")]
    first, second = od.dion_adamw_state(z, bits=8)
    od.dion_adamw_step(od.dion_adamw_plan(z, [torch.zeros(256, device="cuda")], first, second), step=1, lr=1e-3)
    assert not second[0].data.view(torch.uint8).any() and not z[0].any()


def test_roots_of_subnormal_second_moments():
    """Gradients of 3e-20 to 1e-17: second moments around and below float32's least normal number, 1.2e-38.

    A v of 9e-43 or more is right to half of 2^-149, 8e-4 of it, and its root to half of that,
    as is the block's largest; rounding up or down moves a value by less than a step, 2^-3 of it."""
    g = torch.logspace(math.log10(3e-20), -17, 1 << 14, device="cuda")         # a block's values differ by 1.1 at most
    p = [torch.zeros_like(g)]
    first, second = od.dion_adamw_state(p, bits=8)
    od.dion_adamw_step(od.dion_adamw_plan(p, [g], first, second), step=1, lr=1e-3)
    want = math.sqrt(1e-3) * g.double()
    assert torch.all((ref.values(second[0], g.numel()) - want).abs() <= (2.0 ** -3 + 2.0 ** -10) * want)


def test_roots_of_large_second_moments():
    """Second moments on both sides of 2^63, where roots are taken in another way, and up to float32's largest: each
    block's values are within 1.3 of each other, and a value is off by less than a step, 2^-3 of it (and 2^-20)."""
    g = torch.logspace(9, 19.2, 1 << 14, device="cuda")
    p = [torch.zeros_like(g)]
    first, second = od.dion_adamw_state(p, bits=8)
    od.dion_adamw_step(od.dion_adamw_plan(p, [g], first, second), step=1, lr=1e-3)
    want = math.sqrt(1e-3) * g.double()
    assert torch.all((ref.values(second[0], g.numel()) - want).abs() <= (2.0 ** -3 + 2.0 ** -20) * want)
    assert torch.all((p[0].double() + 1e-3).abs() <= 1e-3 * 20 * EPS32)


def test_roots_follow_a_change_that_is_smaller_than_a_step():
    """With gradients of a tenth, r falls by 0.05 % a step; rounded to nearest it would stay where it was.

    Rounding without bias keeps the mean, r <- sqrt(beta2) r being linear (the gradients'
    own part is 0.3 % here).  A value's variance is at most the sum of fall * step, with
    steps of at most 1/8 and a fall of 0.22 in all: 0.17^2, so the mean of 4080 values
    stands within 0.0027; five of these, relative to what is left (0.78), and the 0.3 %."""
    n = 4096
    p, g = [torch.zeros(n, device="cuda")], [torch.full((n,), 1e-4, device="cuda")]
    g[0][::256] = 1e-3                                   # keeps the blocks' scales
    first, second = od.dion_adamw_state(p, bits=8)
    second[0].scale.fill_(1e-3 / 448)
    second[0].data.copy_(torch.full((n,), 448.0, device="cuda").to(torch.float8_e4m3fn))
    plan = od.dion_adamw_plan(p, g, first, second)
    for t in range(1, 501):
        od.dion_adamw_step(plan, step=t, lr=0.0)
    want = math.sqrt(0.999 ** 500 * 1e-6 + (1 - 0.999 ** 500) * 1e-8)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[::256] = False
    mean = float(ref.values(second[0], n)[keep].mean())
    assert abs(mean / want - 1) < 0.021


@pytest.mark.parametrize("bits", [32, 8])
def test_device_scale_skips_and_scales(bits):
    parts = make([5000], BF16, F32, bits)
    before = [copy_of(x) for x in parts[0]], [copy_of(x) for x in parts[2]], [copy_of(x) for x in parts[3]]
    plan = od.dion_adamw_plan(*parts[:4])
    od.dion_adamw_step(plan, step=2, lr=1e-3, grad_scale=torch.tensor([math.nan], device="cuda"))
    flat = lambda x: (x.data.view(torch.uint8), x.scale) if isinstance(x, od.State8) else (x,)  # noqa: E731
    for old, new in zip((*before[0], *before[1], *before[2]), (*parts[0], *parts[2], *parts[3])):
        assert all(torch.equal(a, b) for a, b in zip(flat(old), flat(new)))
    od.dion_adamw_step(plan, step=2, lr=1e-3, grad_scale=torch.tensor([0.25], device="cuda"))
    check(parts, before, 2, scale=0.25)


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step_follows_the_device(bits):
    """A graph of norm and step, replayed with other gradients, rate and count, against calls with numbers."""
    a, b = make([3001, 64], F32, BF16, bits), make([3001, 64], F32, BF16, bits)
    hyper = torch.tensor([1e-3, 0.9, 0.999, 1e-8, 0.1], dtype=torch.float64, device="cuda")
    count = torch.zeros(1, dtype=torch.int64, device="cuda")
    plan, other = od.dion_adamw_plan(*a[:4]), od.dion_adamw_plan(*b[:4])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        od.dion_grad_norm(plan, max_norm=0.01)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = od.dion_grad_norm(plan, max_norm=0.01)
        od.dion_adamw_step(plan, step=count, hyper=hyper, grad_scale=norm[1:], seed=3)
    for t in range(1, 4):
        for x, y in zip(a[1], b[1]):
            x.copy_(torch.randn(x.shape, device="cuda") * 1e-3 * t)
            y.copy_(x)
        hyper[0] = 1e-3 / t
        graph.replay()
        n = od.dion_grad_norm(other, max_norm=0.01)
        od.dion_adamw_step(other, step=t, lr=1e-3 / t, weight_decay=0.1, grad_scale=n[1:], seed=3)
        for x, y in zip((*a[0], *a[2], *a[3]), (*b[0], *b[2], *b[3])):
            x, y = (z.data.view(torch.uint8) if isinstance(z, od.State8) else z for z in (x, y))
            assert torch.equal(x, y)
    assert int(count) == 3
    a[1][0][0] = math.inf
    held = [x.clone() for x in a[0]]
    graph.replay()
    assert int(count) == 3 and all(torch.equal(x, y) for x, y in zip(held, a[0]))       # skipped, and not counted


def test_same_bits_every_time_and_on_any_stream():
    runs = []
    for stream in (None, torch.cuda.Stream()):
        parts = make([100003, 17], BF16, BF16, 8)
        plan = od.dion_adamw_plan(*parts[:4])
        torch.cuda.synchronize()
        norm = od.dion_grad_norm(plan, max_norm=0.1, stream=stream)
        od.dion_adamw_step(plan, step=4, lr=1e-3, grad_scale=norm[1:], stream=stream)
        torch.cuda.synchronize()
        runs.append([norm, *parts[0], *(x.data.view(torch.uint8) for x in parts[2] + parts[3])])
    assert all(torch.equal(x, y) for x, y in zip(*runs))


def test_more_values_than_32_bits_count():
    """The end of a tensor of 2^32 + 777 values."""
    n, k = (1 << 32) + 777, 1500
    p, g = torch.zeros(n, dtype=BF16, device="cuda"), torch.zeros(n, dtype=BF16, device="cuda")
    tail = torch.randn(k, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda") * 1e-3
    g[-k:] = tail.to(BF16)
    first, second = od.dion_adamw_state([p], bits=8)
    od.dion_adamw_step(od.dion_adamw_plan([p], [g], first, second), step=1, lr=1e-2, seed=1)
    start = n - k
    zero = torch.zeros(k, device="cuda").double()
    want, m1, v1, _ = ref.step(zero, g[-k:], zero, zero, 1, lr=1e-2)
    whole = -(-start // 256) * 256                       # the tail's first whole block
    cut = whole - start
    part = lambda s: od.State8(s.data[whole:], s.scale[whole // 256:])  # noqa: E731
    ref.check8(part(first[0]), m1[cut:])
    ref.check8(part(second[0]), v1[cut:].sqrt(), ref.dither(k - cut, 1, 1, 0, start=whole))
    assert torch.all((p[-k:].double() - want).abs() <= (2.0 ** -8 + 20 * EPS32) * want.abs())
    assert not p[:1 << 20].any() and not p[(1 << 31):(1 << 31) + (1 << 20)].any()
    norm = od.dion_grad_norm(od.dion_grad_list([g]))
    want = float(g[-k:].double().norm())
    assert abs(float(norm[0]) - want) <= 2.0 ** -22 * want


# ------------------------------------------------------------------- norm
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("sizes", [[1], [5, 0, 2048], SIZES, [40] * 256, [40] * 383, [40] * 900, [1 << 20], [(1 << 20) + 1], [3_000_001]])
def test_norm(dtype, offset, sizes):
    """Squares and at most 32 sums of them in float32 (rounded the same way at worst): 33 half steps of the sum, half of that of its root."""
    grads = make(sizes, g=dtype, offset=offset)[1]
    want = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    for max_norm in (want / 3, want * 3, math.inf):
        norm, factor = od.dion_grad_norm(od.dion_grad_list(grads), max_norm=max_norm).tolist()
        assert abs(norm - want) <= 18 * EPS32 * want
        assert abs(factor - min(1.0, max_norm / (want + 1e-6))) <= 20 * EPS32


def test_norm_of_nothing_and_of_what_is_not_finite():
    assert od.dion_grad_norm(od.dion_grad_list([])).tolist() == [0.0, 1.0]
    assert od.dion_grad_norm(od.dion_grad_list([torch.empty(0, device="cuda")]), max_norm=2.0).tolist() == [0.0, 1.0]
    for bad in (math.inf, -math.inf, math.nan):
        g = torch.ones(10000, device="cuda")
        g[9999] = bad
        norm, factor = od.dion_grad_norm(od.dion_grad_list([g]), max_norm=1.0).tolist()
        assert not math.isfinite(norm) and math.isnan(factor)


def test_norm_into_given_memory_and_refusals():
    g = [torch.randn(1000, device="cuda")]
    grads = od.dion_grad_list(g)
    large = od.dion_grad_list([torch.randn(1 << 21, device="cuda")])
    out, ws = torch.empty(2, device="cuda"), torch.empty(od.dion_grad_norm_workspace_size(1), dtype=torch.uint8, device="cuda")
    assert od.dion_grad_norm(grads, out=out, workspace=ws) is out
    assert torch.equal(out, od.dion_grad_norm(grads))
    with pytest.raises(ValueError, match="out"):
        od.dion_grad_norm(grads, out=torch.empty(3, device="cuda"))
    with pytest.raises(od.DionError):
        od.dion_grad_norm(large, workspace=ws[:8])
    assert torch.equal(od.dion_grad_norm(large, workspace=torch.empty(od.dion_grad_norm_workspace_size(1), dtype=torch.uint8, device="cuda")),
                       od.dion_grad_norm(large))
    with pytest.raises(od.DionError):
        od.dion_grad_norm(grads, max_norm=0.0)


def test_step_refusals():
    parts = make([100])
    plan = od.dion_adamw_plan(*parts[:4])
    with pytest.raises(ValueError, match="lr"):
        od.dion_adamw_step(plan, step=1)
    with pytest.raises(od.DionError):
        od.dion_adamw_step(plan, step=0, lr=1e-3)
    with pytest.raises(ValueError, match="grad_scale"):
        od.dion_adamw_step(plan, step=1, lr=1e-3, grad_scale=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError, match="hyper"):
        od.dion_adamw_step(plan, step=torch.zeros(1, dtype=torch.int64, device="cuda"), hyper=torch.zeros(5, device="cuda"))
    with pytest.raises(ValueError, match="step"):
        od.dion_adamw_step(plan, step=1, hyper=torch.zeros(5, dtype=torch.float64, device="cuda"))
    with pytest.raises(TypeError, match="plan"):
        od.dion_adamw_step(od.dion_grad_list(parts[1]), step=1, lr=1e-3)
    with pytest.raises(ValueError, match="expected cuda|is on cpu"):
        od.dion_adamw_plan([parts[0][0].cpu()], *parts[1:4])
