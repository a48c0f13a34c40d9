"""4-bit weights: bits of the quantization, values, and products against float64."""
import math

import pytest
import torch

import orthonormal_optimizer_step_gb300 as od
import q4_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def matrix(n, k, dtype=BF16, seed=0, std=0.02):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(n, k, generator=g, device="cuda") * std).to(dtype)


def strided(x, pitch, offset):
    """x as columns of a wider allocation full of NaN."""
    rows, cols = x.shape
    held = torch.full((rows * pitch + offset,), math.nan, device="cuda").to(x.dtype)
    out = held[offset:].view(rows, pitch)[:, :cols]
    out.copy_(x)
    return out


# ------------------------------------------------------------- quantization
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,k", [(1, 1), (3, 31), (5, 128), (7, 129), (2, 250), (17, 1000), (33, 4096), (1000, 65)])
def test_quantize(group, dtype, n, k):
    x = matrix(n, k, dtype)
    for src in (x, strided(x, k + 3, 1)):
        w = od.dion_q4_quantize(src, group=group)
        q, s = ref.groups(x, group)
        assert torch.equal(w.scale.cpu(), s)
        assert torch.equal(w.data.cpu(), ref.pack(q))
        for out in (F32, BF16):
            want = (q.double() * s.double().repeat_interleave(group, 1)[:, :k]).to(F32).to(out)
            assert torch.equal(od.dion_q4_dequantize(w, out_dtype=out).cpu(), want)


def test_quantize_ties_and_extremes():
    """Quotients half-way between whole numbers, groups of zeros, of subnormals, of the largest values."""
    x = torch.zeros(8, 128, device="cuda")
    x[0] = torch.arange(128, device="cuda") % 15 / 2 - 3.5
    x[0, 0] = 7.0                                        # scale 1: halves are ties
    x[1] = -x[0]
    x[2] = 1e-42
    x[2, 5] = -3e-41
    x[3] = 3e38
    x[3, 7] = -3.3e38
    x[4] = 2.0 ** -133                                   # the scale, a seventh of it, rounds to zero
    x[5] = torch.linspace(-1, 1, 128, device="cuda")
    x[6, 3] = 1e-30
    for group in (32, 64, 128):
        w = od.dion_q4_quantize(x, group=group)
        q, s = ref.groups(x, group)
        assert torch.equal(w.scale.cpu(), s) and torch.equal(w.data.cpu(), ref.pack(q))


def test_quantize_marks_groups_that_are_not_finite():
    x = matrix(4, 300, F32)
    x[0, 5], x[1, 140], x[2, 299] = math.inf, math.nan, -math.inf
    for group in (32, 128):
        w = od.dion_q4_quantize(x, group=group)
        q, s = ref.groups(x, group)
        assert torch.equal(torch.isnan(w.scale.cpu()), torch.isnan(s)) and torch.isnan(s).sum() == 3
        assert torch.equal(w.data.cpu(), ref.pack(q))
        bad = torch.isnan(s).repeat_interleave(group, 1)[:, :300]
        assert torch.equal(torch.isnan(od.dion_q4_dequantize(w).cpu()), bad)
        y = od.dion_q4_matmul(torch.ones(1, 300, device="cuda", dtype=BF16), w)[0]
        assert torch.isnan(y[:3]).all() and torch.isfinite(y[3])


def test_quantize_into_given_memory():
    x = matrix(9, 200)
    data = torch.full((9, 192), 7, dtype=torch.uint8, device="cuda")
    scale = torch.full((9, 5), 3.0, dtype=BF16, device="cuda")
    out = od.Q4(data[:, :128], scale[:, :2], 200, 128)
    assert od.dion_q4_quantize(x, group=128, out=out) is out
    new = od.dion_q4_quantize(x, group=128)
    assert torch.equal(out.data, new.data) and torch.equal(out.scale, new.scale)
    assert (data[:, 128:] == 7).all() and (scale[:, 2:] == 3).all()
    y = torch.zeros(9, 300, device="cuda")
    assert torch.equal(od.dion_q4_dequantize(out, out=y[:, 50:250]), od.dion_q4_dequantize(new, out_dtype=F32))
    assert not y[:, :50].any() and not y[:, 250:].any()
    with pytest.raises(ValueError, match="groups of"):
        od.dion_q4_quantize(x, group=64, out=out)
    with pytest.raises(ValueError, match="rows, cols"):
        od.dion_q4_quantize(x[0])
    with pytest.raises(TypeError):
        od.dion_q4_quantize(x.half())


# ------------------------------------------------------------------ products
def values(w):
    q = ref.unpack(w.data, w.cols)[:, :w.cols].double().cuda()
    return q * w.scale.double().repeat_interleave(w.group, 1)[:, :w.cols]


def x_values(x):
    if not isinstance(x, od.Q8):
        return x.double().reshape(-1, x.shape[-1])
    s = torch.exp2(x.scale.view(torch.uint8).double() - 127).repeat_interleave(128, 1)[:, :x.data.shape[1]]
    return x.data.double() * s


def check(y, x, w):
    """Products are exact but for x's own part (float32: 2^-24 of a value; values far below the largest of a
    row's 128 columns: 2^-39 of that).  A chain of sums is at most the share's products of the tensor cores (16
    terms each, truncated: 2^-23), its groups, chunks, the shares and the terms; the result is rounded once."""
    xv, wv = x_values(x), values(w)
    want = xv @ wv.t()
    size = xv.abs() @ wv.abs().t()
    k = w.cols
    chain = k / 16 + k / w.group + k / 128 + 8 + 8
    far = 2.0 ** -39 * k * xv.nan_to_num().abs().amax(1, keepdim=True) * wv.nan_to_num().abs().amax(1)
    slack = (chain * 2.0 ** -23 + 2.0 ** -24) * size + far + (2.0 ** -8 * want.abs() if y.dtype is BF16 else 2.0 ** -24 * want.abs())
    got = y.double().reshape(want.shape)
    assert torch.all((got - want).abs() <= slack)
    if y.dtype is F32 and want.numel() >= 64:
        # in the mean square rounding errors add like a walk: sqrt(chain) of the worst, of a typical sum's size
        rms = (xv.square() @ wv.t().square()).sqrt()
        assert float((got - want).square().mean().sqrt()) <= 4 * math.sqrt(chain) * 2.0 ** -23 * float(rms.square().mean().sqrt())


def rows(m, k, kind, seed=1):
    x = matrix(m, k, BF16 if kind == "bf16" else F32, seed, 1.0)
    if kind in ("bf16", "f32"):
        return x
    return od.dion_q8_quantize(x, dtype=torch.float8_e4m3fn if kind == "e4m3" else torch.float8_e5m2)[0]


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3", "e5m2"])
@pytest.mark.parametrize("m", [1, 2, 5, 8, 9, 16, 17, 32, 33, 70])
@pytest.mark.parametrize("n,k,group", [(1, 1, 32), (16, 127, 64), (63, 128, 128), (65, 129, 32), (200, 1000, 64),
                                       (130, 4096, 128), (1000, 520, 32), (64, 20000, 128)])
def test_matmul(kind, m, n, k, group):
    w = od.dion_q4_quantize(matrix(n, k), group=group)
    x = rows(m, k, kind)
    for out in (BF16, F32):
        check(od.dion_q4_matmul(x, w, out_dtype=out), x, w)


@pytest.mark.parametrize("n,k", [(4096, 4096), (14336, 4096), (4096, 14336), (20000, 640), (128, 65536)])
@pytest.mark.parametrize("m", [1, 16])
def test_matmul_of_real_sizes(n, k, m):
    w = od.dion_q4_quantize(matrix(n, k), group=128)
    for kind in ("bf16", "e4m3", "f32"):
        x = rows(m, k, kind)
        check(od.dion_q4_matmul(x, w, out_dtype=F32), x, w)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_strides_and_alignment(kind):
    """Rows of wider allocations at odd places, scales of odd pitch, an output between other columns; what lies beside stays."""
    for group, pad in ((32, 1), (64, 3), (128, 5)):
        w = od.dion_q4_quantize(matrix(100, 1000), group=group)
        wide = torch.zeros(100, w.data.shape[1] + 16, dtype=torch.uint8, device="cuda")
        scale = torch.full((100, w.scale.shape[1] + pad), math.nan, dtype=BF16, device="cuda")
        wide[:, :-16], scale[:, :-pad] = w.data, w.scale
        v = od.Q4(wide[:, :-16], scale[:, :-pad], 1000, group)
        x = rows(5, 1000, kind)
        for src in (x, strided(x, 1003, 1), strided(x, 1004, 0)):
            y = torch.full((5, 150), 7.0, device="cuda")
            od.dion_q4_matmul(src, v, out=y[:, 20:120])
            assert torch.equal(y[:, 20:120], od.dion_q4_matmul(x, w, out_dtype=F32))
            assert (y[:, :20] == 7).all() and (y[:, 120:] == 7).all()


def test_leading_dimensions_and_empty():
    w = od.dion_q4_quantize(matrix(48, 256))
    x = matrix(6, 256, seed=2, std=1.0)
    y = od.dion_q4_matmul(x, w)
    assert torch.equal(od.dion_q4_matmul(x.view(2, 3, 256), w), y.view(2, 3, 48))
    assert od.dion_q4_matmul(x[:0], w).shape == (0, 48)
    assert od.dion_q4_matmul(x, od.new_q4(0, 256)).shape == (6, 0)
    none = od.dion_q4_quantize(torch.empty(48, 0, device="cuda"))
    assert none.data.shape == (48, 0) and od.dion_q4_dequantize(none).shape == (48, 0)
    assert not od.dion_q4_matmul(torch.empty(6, 0, device="cuda"), none, out=torch.ones(6, 48, device="cuda")).any()


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3"])
def test_a_bad_row_stays_alone(kind):
    w = od.dion_q4_quantize(matrix(70, 600))
    x = matrix(11, 600, BF16 if kind == "bf16" else F32, 1, 1.0)
    good = x.clone()
    x[3, 77], x[7, 500] = math.inf, math.nan
    if kind == "e4m3":
        x, good = od.dion_q8_quantize(x)[0], od.dion_q8_quantize(good)[0]
    y, z = od.dion_q4_matmul(x, w, out_dtype=F32), od.dion_q4_matmul(good, w, out_dtype=F32)
    keep = [i for i in range(11) if i not in (3, 7)]
    assert torch.equal(y[keep], z[keep]) and torch.isnan(y[7]).all()
    column = values(w)[:, 77]
    if kind == "e4m3":                                   # infinities are NaN there
        assert torch.isnan(y[3]).all()
    else:                                                # infinity times zero is NaN
        assert torch.equal(torch.isnan(y[3]), column == 0) and torch.equal(y[3] == math.inf, column > 0)


def test_same_bits_captured_on_streams_and_at_once():
    w = [od.dion_q4_quantize(matrix(2000, 4096, seed=i), group=64) for i in range(2)]
    x = [matrix(3, 4096, seed=5 + i, std=1.0) for i in range(2)]
    y = [od.dion_q4_matmul(x[i], w[i]) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        z = [od.dion_q4_matmul(x[i], w[i], stream=streams[i]) for i in range(2)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(y, z))
    out = torch.empty_like(y[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = od.dion_q4_quantize(od.dion_q4_dequantize(w[0]), group=64)
        od.dion_q4_matmul(x[0], w[0], out=out)
    x[0].copy_(x[1])
    graph.replay()
    assert torch.equal(out, od.dion_q4_matmul(x[1], w[0]))
    assert torch.equal(q.data, od.dion_q4_quantize(od.dion_q4_dequantize(w[0]), group=64).data)


def test_large_matrix_offsets():
    """Data beyond 2^32 bytes: the last rows of 600000 x 16384."""
    n, k = 600000, 16384
    w = od.new_q4(n, k)
    w.data.fill_(0x88)
    w.scale.fill_(1.0)
    last = od.dion_q4_quantize(matrix(100, k))
    w.data[-100:], w.scale[-100:] = last.data, last.scale
    x = matrix(2, k, seed=3, std=1.0)
    y = od.dion_q4_matmul(x, w)
    assert torch.equal(y[:, -100:], od.dion_q4_matmul(x, last)) and not y[:, :-100].any()
    part = torch.empty(n, k, dtype=BF16, device="cuda")
    od.dion_q4_dequantize(w, out=part)
    assert torch.equal(part[-100:], od.dion_q4_dequantize(last)) and not part[1 << 18].any()
    again = od.dion_q4_quantize(part)
    assert torch.equal(again.data[-100:], od.dion_q4_quantize(part[-100:]).data) and (again.data[1 << 18] == 0x88).all()


def test_matmul_refusals():
    w = od.dion_q4_quantize(matrix(48, 256))
    x = matrix(3, 256)
    with pytest.raises(ValueError, match="columns"):
        od.dion_q4_matmul(x[:, :255], w)
    with pytest.raises(ValueError, match="contiguous rows"):
        od.dion_q4_matmul(matrix(256, 3).t(), w)
    with pytest.raises(TypeError):
        od.dion_q4_matmul(x.half(), w)
    with pytest.raises(TypeError):
        od.dion_q4_matmul(x, w, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="out must be"):
        od.dion_q4_matmul(x, w, out=torch.empty(3, 47, device="cuda"))
    with pytest.raises(ValueError, match="scale for each 128"):
        od.dion_q4_matmul(od.dion_q8_quantize(x, square=True)[0], w)
    with pytest.raises(ValueError, match="at least two"):
        od.dion_q4_matmul(x[0], w)
    y = od.dion_q4_matmul(x.clone().requires_grad_(), w)
    with pytest.raises(NotImplementedError, match="no derivative"):
        y.float().sum().backward()


def test_every_call_checks_the_device(monkeypatch):
    from orthonormal_optimizer_step_gb300 import adamw, q8
    x = matrix(3, 256)
    w = od.dion_q4_quantize(x)
    grads = od.dion_grad_list([x])
    monkeypatch.setattr(q8, "_current_device", lambda: x.get_device() + 1)
    monkeypatch.setattr(adamw, "_current_device", lambda: x.get_device() + 1)
    for call in (lambda: od.dion_q4_quantize(x), lambda: od.dion_q4_dequantize(w), lambda: od.dion_q4_matmul(x, w),
                 lambda: od.dion_grad_norm(grads), lambda: od.dion_grad_list([x])):
        with pytest.raises(ValueError, match="current device"):
            call()
