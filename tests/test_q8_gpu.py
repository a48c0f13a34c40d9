"""The 8-bit linear layer's operators against plain 64-bit implementations.

Tolerances:
  quantize    none: maxima, power-of-two scales and the divisions by them are
              exact, and each value is rounded once to nearest even.
  matmul      the tensor core adds the 32 products of an instruction and the
              running sum in at least 24 bits: at most K/32 + 32 roundings of
              magnitudes up to S = sum |a b|, each 2^-23 at worst, so
              (K/32 + 32) 2^-23 S, plus the rounding to bfloat16 (2^-8 of C).
  norm        h exactly.  A thread adds at most 64 squares and joins take at
              most 12 more additions, each 2^-24, halved by the square root,
              plus division, root and mean: 42 * 2^-24 for rstd; two more
              products for y: TOL_Y = 45 * 2^-24.
  backward    as many operations as the forward pass for the mean, so
              TAU = 100 * 2^-24 of the terms' magnitudes, plus the rounding to
              bfloat16; dw: one rounding a row and two a product, (rows + 8) 2^-24
              of the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

import orthonormal_optimizer_step_gb300 as od
import q8_ref as ref

pytestmark = pytest.mark.gpu

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
BF16, F32 = torch.bfloat16, torch.float32
TOL_RSTD, TOL_Y, TAU = 42 * 2.0 ** -24, 45 * 2.0 ** -24, 100 * 2.0 ** -24


def randn(*shape, seed=0, std=1.0, dtype=F32, spread=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 17 * sum(shape))
    t = torch.randn(shape, generator=g, device="cuda") * std
    if spread:
        t = t * torch.exp(spread * torch.randn(shape[-1], generator=g, device="cuda"))
    return t.to(dtype)


def same_q8(q, x, dtype, square):
    """q is exactly the quantization of the float64 matrix x."""
    want, e = ref.quantize(x, dtype, square)
    assert np.array_equal(ref.exponents(q.scale), e)
    assert np.array_equal(ref.f64(q.data), want, equal_nan=True)


def rounding(c, dtype):
    return np.abs(c) * (2.0 ** -8 if dtype == BF16 else 2.0 ** -24)


# ----------------------------------------------------------------- quantize
@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (4096, 1), (128, 128), (129, 127), (7, 250), (300, 1000),
                                       (513, 392), (130, 2049)])
def test_quantize(rows, cols, square, dtype, fmt):
    x = randn(rows, cols, dtype=dtype, std=1e-3, spread=2.0)
    both = od.dion_q8_quantize(x, form="both", square=square, dtype=fmt)
    same_q8(both[0], ref.f64(x), fmt, square)
    same_q8(both[1], ref.f64(x).T, fmt, square)
    one, none = od.dion_q8_quantize(x, square=square, dtype=fmt)
    assert none is None
    same_q8(one, ref.f64(x), fmt, square)
    none, one = od.dion_q8_quantize(x, form="cols", square=square, dtype=fmt)
    assert none is None
    same_q8(one, ref.f64(x).T, fmt, square)


def special(dtype):
    """Blocks whose largest magnitude is at, just under and just over the format's
    edge, zero, subnormal, the largest float, and non-finite."""
    x = torch.zeros(140, 400)
    for i, a in enumerate([448.0, 448.0 * 2.0 ** -9, 57344.0, 449.0, 447.0, 450.0, 1.75, 1.7578125, 3.3e38, -3.3e38,
                           2.0 ** -126, 2.0 ** -133, 1e-40, 0.0, -0.0, 3.0 * 2.0 ** -130]):
        x[i, :128] = a * torch.linspace(-1, 1, 128)
        x[i, 200] = a
        x[i, 300] = a / 3
    x[20, 5], x[21, 140], x[22, 390], x[23, :] = float("inf"), -float("inf"), float("nan"), float("nan")
    x[20, 6:20] = 3.0
    x[139, 399] = 7.0
    return x.to(dtype)


@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("square", [False, True])
def test_quantize_special_values(square, dtype, fmt):
    x = special(dtype)
    r, c = od.dion_q8_quantize(x.cuda(), form="both", square=square, dtype=fmt)
    v = x.double().numpy()
    same_q8(r, v, fmt, square)
    same_q8(c, v.T, fmt, square)


def test_quantize_strides_batch_and_offsets():
    base = randn(3, 70, 333, seed=2)
    for x in (base[:, :, 1:300], base[:, 2:69, :], base[1:, ::2, 4:204], base[:, :, 5:6]):
        for square in (False, True):
            r, c = od.dion_q8_quantize(x, form="both", square=square)
            for b in range(x.shape[0]):
                same_q8(od.Q8(r.data[b], r.scale[b]), ref.f64(x[b]), E4M3, square)
                same_q8(od.Q8(c.data[b], c.scale[b]), ref.f64(x[b]).T, E4M3, square)
    # row offsets past 2^31 elements
    big = torch.empty((1 << 31) + 4096, dtype=BF16, device="cuda")
    x = big.as_strided((2, 300), (1 << 31, 1))
    x.copy_(randn(2, 300, dtype=BF16, seed=5))
    r, c = od.dion_q8_quantize(x, form="both")
    same_q8(r, ref.f64(x), E4M3, False)
    same_q8(c, ref.f64(x).T, E4M3, False)


def test_quantize_empty():
    for rows, cols in ((0, 256), (256, 0)):
        r, c = od.dion_q8_quantize(torch.empty(rows, cols, device="cuda"), form="both")
        assert r.data.shape == (rows, cols) and c.data.shape == (cols, rows)
    r, _ = od.dion_q8_quantize(torch.empty(0, 4, 4, device="cuda"))
    assert r.data.shape == (0, 4, 4)


def test_quantize_writes_only_its_elements():
    x = randn(130, 200, seed=3)
    data = torch.full((200, 176), 0x55, dtype=torch.uint8, device="cuda")
    scale = torch.full((200, 8), 0x55, dtype=torch.uint8, device="cuda")
    out = od.Q8(data.view(E4M3)[:, :130], scale.view(torch.float8_e8m0fnu)[:, :2])
    od.dion_q8_quantize(x, form="cols", out=(None, out))
    same_q8(out, ref.f64(x).T, E4M3, False)
    assert bool((data[:, 130:] == 0x55).all()) and bool((scale[:, 2:] == 0x55).all())


@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("rows,cols", [(1, 64), (200, 500), (129, 1024)])
def test_quantize_normed(rows, cols, dtype, wdtype):
    x, w = randn(rows, cols, dtype=dtype), (1 + 0.2 * randn(cols, seed=4)).to(wdtype)
    rstd = torch.rand(rows, device="cuda") + 0.5
    y = (x.float().cpu().numpy() * rstd.cpu().numpy()[:, None]) * w.float().cpu().numpy()   # float32, as defined
    assert y.dtype == np.float32
    r, c = od.dion_q8_quantize(x, form="both", rstd=rstd, weight=w)
    same_q8(r, y.astype(np.float64), E4M3, False)
    same_q8(c, y.astype(np.float64).T, E4M3, False)


# ------------------------------------------------------------------- matmul
def q8_operand(rows, k, fmt=E4M3, square=False, seed=0):
    q, _ = od.dion_q8_quantize(randn(rows, k, seed=seed, spread=1.0), square=square, dtype=fmt)
    return q


def check_matmul(a, b, out_dtype, c=None):
    va, vb = ref.values(a), ref.values(b)
    if c is None:
        c = od.dion_q8_matmul(a, b, out_dtype=out_dtype)
    torch.cuda.synchronize()
    assert od.dion_q8_status() == 0
    assert c.shape == (va.shape[0], vb.shape[0]) and c.dtype == out_dtype
    want, size = va @ vb.T, np.abs(va) @ np.abs(vb).T
    k = va.shape[1]
    err = np.abs(ref.f64(c) - want)
    assert np.all(err <= (k / 32 + 32) * 2.0 ** -23 * size + rounding(want, out_dtype)), err.max()


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 33, 64, 65, 128, 129, 300])
@pytest.mark.parametrize("n,k", [(1, 1), (128, 128), (127, 129), (200, 500), (513, 1000), (256, 2064), (1111, 640)])
def test_matmul_sizes(m, n, k):
    check_matmul(q8_operand(m, k), q8_operand(n, k, square=True, seed=1), BF16)
    check_matmul(q8_operand(m, k, fmt=E5M2), q8_operand(n, k, seed=1), F32)


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("m,n,k", [(512, 768, 768), (1024, 2304, 768), (257, 4096, 4096), (1000, 1500, 8200),
                                   (2048, 2048, 256), (5, 4096, 14336), (200, 4000, 8300), (256, 3500, 8192), (1000, 6144, 2000),
                                   (2048, 4608, 1030), (100, 64, 16384), (3000, 40, 128)])
def test_matmul_larger(m, n, k, out_dtype):
    check_matmul(q8_operand(m, k, square=True), q8_operand(n, k, square=True, seed=1), out_dtype)
    check_matmul(q8_operand(m, k), q8_operand(n, k, seed=1), out_dtype)


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("m,n,k", [(395, 4984, 2000), (601, 5632, 4000), (397, 4865, 4000), (1001, 4104, 4100)])
def test_matmul_pairs(m, n, k, out_dtype):
    """Sizes that CTA pairs take (224 and 256 wide, and 256 wide with C's rows
    unaligned), whole and into a part of a larger matrix."""
    a, b = q8_operand(m, k, fmt=E5M2), q8_operand(n, k, square=True, seed=1)
    va, vb = (torch.from_numpy(ref.values(q)).cuda() for q in (a, b))
    want, size = (va @ vb.T).cpu().numpy(), (va.abs() @ vb.abs().T).cpu().numpy()
    big = torch.full((m + 2, n + 24), 7.0, dtype=out_dtype, device="cuda")
    with od.profile() as p:
        c = od.dion_q8_matmul(a, b, out_dtype=out_dtype)
        od.dion_q8_matmul(a, b, out=big[1:m + 1, 8:8 + n])
    torch.cuda.synchronize()
    assert od.dion_q8_status() == 0
    assert set(p.read()) == {"q8_matmul_pair"}
    tol = (k / 32 + 32) * 2.0 ** -23 * size + rounding(want, out_dtype)
    assert np.all(np.abs(ref.f64(c) - want) <= tol)
    assert torch.equal(big[1:m + 1, 8:8 + n], c)
    big[1:m + 1, 8:8 + n] = 7.0
    assert bool((big == 7).all())


@pytest.mark.parametrize("af", [E4M3, E5M2])
@pytest.mark.parametrize("bf", [E4M3, E5M2])
def test_matmul_formats(af, bf):
    for m in (3, 200):
        check_matmul(q8_operand(m, 700, fmt=af), q8_operand(150, 700, fmt=bf, seed=1), F32)


def test_matmul_every_scale_is_used():
    """Scales that differ wildly between rows and blocks: each block's products carry their own."""
    for m in (4, 150, 400):
        a, b = q8_operand(m, 1300), q8_operand(300, 1300, seed=1)
        for q, s in ((a, 5), (b, 6)):
            g = torch.Generator(device="cuda")
            g.manual_seed(s)
            q.scale.view(torch.uint8).copy_(torch.randint(107, 148, q.scale.shape, generator=g, device="cuda"))
        check_matmul(a, b, F32)


def test_matmul_extreme_scales():
    a, b = q8_operand(20, 128), q8_operand(30, 128, seed=1)
    a.scale.view(torch.uint8).fill_(0)             # 2^-127
    b.scale.view(torch.uint8).fill_(254)           # 2^127
    check_matmul(a, b, F32)


@pytest.mark.parametrize("m", [5, 100, 600])
def test_matmul_nan_stays_in_its_row(m):
    k = 400
    for which in ("value", "scale"):
        a, b = q8_operand(m, k), q8_operand(290, k, seed=1)
        clean = od.dion_q8_matmul(a, b)
        if which == "value":
            a.data.view(torch.uint8)[3, 130] = 0x7f
            b.data.view(torch.uint8)[7, 399] = 0x7f
        else:
            a.scale.view(torch.uint8)[3, 1] = 255
            b.scale.view(torch.uint8)[7, 3] = 255
        c = od.dion_q8_matmul(a, b)
        bad = torch.zeros_like(c, dtype=torch.bool)
        bad[3], bad[:, 7] = True, True
        assert torch.equal(torch.isnan(c), bad)
        assert torch.equal(c[~bad], clean[~bad])


def test_matmul_zero_contraction_and_empty():
    c = torch.full((5, 300), 7.0, device="cuda")
    od.dion_q8_matmul(od.new_q8(5, 0), od.new_q8(300, 0), out=c)
    assert bool((c == 0).all())
    view = torch.full((5, 300), 7.0, dtype=BF16, device="cuda")
    od.dion_q8_matmul(od.new_q8(5, 0), od.new_q8(200, 0), out=view[:, 50:250])
    assert bool((view[:, 50:250] == 0).all()) and bool((view[:, :50] == 7).all()) and bool((view[:, 250:] == 7).all())
    assert od.dion_q8_matmul(od.new_q8(0, 256), od.new_q8(3, 256)).shape == (0, 3)
    assert od.dion_q8_matmul(od.new_q8(4, 256), od.new_q8(0, 256)).shape == (4, 0)


@pytest.mark.parametrize("m,n", [(3, 131), (70, 131), (300, 131), (600, 1031)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_matmul_writes_only_its_elements(m, n, dtype):
    a, b = q8_operand(m, 300), q8_operand(n, 300, seed=1)
    for off in (0, 1, 2, 8):
        big = torch.full((m + 2, n + 21), 7.0, dtype=dtype, device="cuda")
        out = big[1:m + 1, off:off + n]
        check_matmul(a, b, dtype, od.dion_q8_matmul(a, b, out=out))
        big[1:m + 1, off:off + n] = 7.0
        assert bool((big == 7).all())


def test_matmul_long_pitches():
    """Operand and output rows more than 2^31 elements apart."""
    m, n, k = 3, 130, 300
    a, b = q8_operand(m, k), q8_operand(n, k, seed=1)
    far = torch.zeros((1 << 31) * (m - 1) + 4096, dtype=torch.uint8, device="cuda").view(E4M3)
    data = far.as_strided((m, k), (1 << 31, 1))
    data.view(torch.uint8).copy_(a.data.view(torch.uint8))
    out = torch.zeros((1 << 31) * (m - 1) + 4096, dtype=BF16, device="cuda").as_strided((m, n), (1 << 31, 1))
    check_matmul(od.Q8(data, a.scale), b, BF16, od.dion_q8_matmul(od.Q8(data, a.scale), b, out=out))


def test_same_bits_every_time():
    a, b = q8_operand(70, 9000), q8_operand(900, 9000, seed=1)
    first = od.dion_q8_matmul(a, b, out_dtype=F32)
    dy, h, w = randn(900, 700), randn(900, 700, seed=1), randn(700, seed=2)
    rstd = torch.rand(900, device="cuda")
    g = od.dion_rms_norm_backward(dy, h, rstd, w)
    for _ in range(20):
        assert torch.equal(first, od.dion_q8_matmul(a, b, out_dtype=F32))
        for u, v in zip(g, od.dion_rms_norm_backward(dy, h, rstd, w)):
            assert torch.equal(u, v)


# --------------------------------------------------------------------- norm
def check_norm(x, r, w, eps, fmt, got):
    q, h, rstd = got
    want_h = x if r is None else (x.float() + r.float()).to(x.dtype)
    assert torch.equal(h, want_h) or torch.equal(torch.isnan(h), torch.isnan(want_h))
    y, want_rstd = ref.norm(ref.f64(want_h), ref.f64(w), eps)
    assert np.all(np.abs(ref.f64(rstd) - want_rstd) <= TOL_RSTD * want_rstd)
    top, bits, low = ref.FORMATS[fmt]
    cols = y.shape[1]
    # a scale may differ from the 64-bit one only where y's rounding moves the block's maximum across the edge
    e = ref.exponents(q.scale)
    assert np.all(e >= ref.block_exponents(y * (1 - TOL_Y), fmt, False))
    assert np.all(e <= ref.block_exponents(y * (1 + TOL_Y), fmt, False))
    s = np.ldexp(1.0, ref.spread(e, *y.shape))
    _, ey = np.frexp(y / s)
    half = np.ldexp(0.5, np.maximum(ey - 1, low) - bits) * s
    assert np.all(np.abs(ref.f64(q.data) * s - y) <= half * (1 + 1e-9) + 2 * TOL_Y * np.abs(y))
    assert q.data.shape == y.shape and cols == w.shape[0]


NORM_SIZES = [(1, 1), (1, 4096), (3, 64), (17, 127), (40, 128), (9, 1000), (33, 1001), (5, 2048), (4, 2056), (6, 8192),
              (3, 16384), (2, 16392), (2, 32768), (2, 33000), (2, 53248)]


@pytest.mark.parametrize("dtype,wdtype,fmt", [(BF16, BF16, E4M3), (F32, F32, E4M3), (BF16, F32, E5M2)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", NORM_SIZES)
def test_norm(rows, cols, residual, dtype, wdtype, fmt):
    x, w = randn(rows, cols, dtype=dtype, spread=0.5), (1 + 0.1 * randn(cols, seed=1)).to(wdtype)
    r = randn(rows, cols, dtype=dtype, seed=2, std=3.0) if residual else None
    check_norm(x, r, w, 1e-6, fmt, od.dion_rms_norm_q8(x, w, residual=r, dtype=fmt))


# rows enough for the kernels that stream them: one, two and four chunks a thread, some of them past the row
STREAM_SIZES = [(5100, 72), (5100, 512), (3100, 1032), (1300, 4096), (1300, 4104), (700, 8192), (340, 16384)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", STREAM_SIZES)
def test_norm_streamed(rows, cols, residual):
    x, w = randn(rows, cols, dtype=BF16, spread=0.5), (1 + 0.1 * randn(cols, seed=1)).to(BF16)
    r = randn(rows, cols, dtype=BF16, seed=2, std=3.0) if residual else None
    x[rows - 1, 3] = float("nan")
    want = od.dion_rms_norm_q8(x[:200], w, residual=None if r is None else r[:200])       # a row a CTA
    with od.profile() as p:
        got = od.dion_rms_norm_q8(x, w, residual=r, h=None if r is None else r.clone())
    torch.cuda.synchronize()
    assert set(p.read()) == {"rms_norm_q8_stream"}
    assert torch.equal(got[1][:200], want[1][:200]) and torch.allclose(got[2][:200], want[2], rtol=TOL_RSTD, atol=0)
    q, h, rstd = got
    assert bool(torch.isnan(q.data[rows - 1].float()).all()) and bool(torch.isnan(rstd[rows - 1]))
    keep = torch.arange(rows, device="cuda") != rows - 1
    check_norm(x[keep], None if r is None else r[keep], w, 1e-6, E4M3, (od.Q8(q.data[keep], q.scale[keep]), h[keep], rstd[keep]))


def test_norm_shapes_strides_and_in_place():
    w = 1 + 0.1 * randn(300, seed=1)
    base = randn(4, 50, 333, dtype=BF16)
    x, r = base[1, :, 1:301], base[2, :, 3:303]
    check_norm(x, r, w, 1e-5, E4M3, od.dion_rms_norm_q8(x, w, residual=r, eps=1e-5))
    x, r = base[1, :40, 8:308], base[2, :40, 16:316]
    for h in ("x", "r"):
        a, b = x.clone(), r.clone()
        got = od.dion_rms_norm_q8(a, w, residual=b, h=a if h == "x" else b)
        assert got[1] is (a if h == "x" else b)
        check_norm(x, r, w, 1e-6, E4M3, got)
    x3 = randn(2, 3, 300)
    q, h, rstd = od.dion_rms_norm_q8(x3, w, residual=x3)
    assert h.shape == x3.shape and q.data.shape == (6, 300) and rstd.shape == (6,)
    q, h, rstd = od.dion_rms_norm_q8(x3, w)
    assert h is x3
    q, _, _ = od.dion_rms_norm_q8(torch.empty(0, 300, device="cuda"), w)
    assert q.data.shape == (0, 300)


def test_norm_and_gradient_long_pitches():
    """Rows more than 2^31 elements apart."""
    far = 1 << 31
    big = torch.empty(2 * far + 4096, dtype=BF16, device="cuda")

    def at(off, seed):
        t = big.as_strided((3, 264), (far, 1), off)
        t.copy_(randn(3, 264, dtype=BF16, seed=seed))
        return t

    x, r, dy = at(0, 1), at(264, 2), at(528, 3)
    h, dx = big.as_strided((3, 264), (far, 1), 800), big.as_strided((3, 264), (far, 1), 1064)
    w = (1 + 0.1 * randn(264, seed=4)).to(BF16)
    got = od.dion_rms_norm_q8(x, w, residual=r, h=h)
    check_norm(x, r, w, 1e-6, E4M3, got)
    check_backward(dy, h, got[2], w, r, od.dion_rms_norm_backward(dy, h, got[2], w, dh=r, dx=dx), BF16)


def test_norm_zero_rows_of_values_and_non_finite_rows():
    x = randn(5, 256)
    x[1], x[2, 7], x[3, 9] = 0.0, float("inf"), float("nan")
    w = torch.ones(256, device="cuda")
    q, _, rstd = od.dion_rms_norm_q8(x, w)
    d = ref.f64(q.data)
    assert np.all(d[1] == 0) and float(rstd[1]) == pytest.approx(1e3, rel=1e-6)
    assert np.isnan(d[2, 7]) and np.all(np.delete(d[2], 7) == 0)      # 1 / sqrt(inf) = 0
    assert np.all(np.isnan(d[3]))
    good = od.dion_rms_norm_q8(x[[0, 4]], w)[0]
    assert np.array_equal(d[[0, 4]], ref.f64(good.data))


# ----------------------------------------------------------------- gradient
def check_backward(dy, h, rstd, w, dh, got, dtype):
    a = [ref.f64(t) for t in (dy, h, rstd, w)]
    d = None if dh is None else ref.f64(dh)
    dx, dw = ref.norm_backward(*a, d)
    xhat = a[1] * a[2][:, None]
    g = a[0] * a[3]
    size = np.abs(a[2])[:, None] * (np.abs(g) + np.abs(xhat) * np.abs(g * xhat).mean(1, keepdims=True))
    size = size + (0 if d is None else np.abs(d))
    assert np.all(np.abs(ref.f64(got[0]) - dx) <= TAU * size + rounding(dx, dtype))
    assert got[1].dtype == F32
    assert np.all(np.abs(ref.f64(got[1]) - dw) <= (dy.shape[0] + 8) * 2.0 ** -24 * np.abs(a[0] * xhat).sum(0))


@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", NORM_SIZES + [(700, 4096), (5000, 64), (1300, 333)])
def test_backward(rows, cols, residual, dtype, wdtype):
    h, w = randn(rows, cols, dtype=dtype, spread=0.5), (1 + 0.1 * randn(cols, seed=1)).to(wdtype)
    dy = randn(rows, cols, dtype=dtype, seed=2, std=0.01)
    dh = randn(rows, cols, dtype=dtype, seed=3, std=0.01) if residual else None
    rstd = 1.0 / torch.sqrt(h.float().square().mean(1) + 1e-6)
    check_backward(dy, h, rstd, w, dh, od.dion_rms_norm_backward(dy, h, rstd, w, dh=dh), dtype)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", STREAM_SIZES)
def test_backward_streamed(rows, cols, residual):
    h, w = randn(rows, cols, dtype=BF16, spread=0.5), (1 + 0.1 * randn(cols, seed=1)).to(BF16)
    dy = randn(rows, cols, dtype=BF16, seed=2, std=0.01)
    dh = randn(rows, cols, dtype=BF16, seed=3, std=0.01) if residual else None
    rstd = 1.0 / torch.sqrt(h.float().square().mean(1) + 1e-6)
    with od.profile() as p:
        got = od.dion_rms_norm_backward(dy, h, rstd, w, dh=dh, dx=None if dh is None else dh.clone())
    torch.cuda.synchronize()
    assert set(p.read()) == {"rms_norm_backward_stream", "rms_norm_backward_sum"}
    check_backward(dy, h, rstd, w, dh, got, BF16)


@pytest.mark.parametrize("rows,cols", [(1, 8192), (2048, 1000), (2048, 1024), (255, 8190), (77, 40), (2049, 100), (300, 8193)])
def test_backward_in_one_launch(rows, cols):
    """Small problems take one kernel and no workspace; in place, or just too
    large, the others; all agree."""
    h, w, dy, dh = randn(rows, cols), 1 + 0.1 * randn(cols, seed=1), randn(rows, cols, seed=2), randn(rows, cols, seed=3)
    rstd = torch.rand(rows, device="cuda") + 0.5
    small = rows <= 2048 and cols <= 8192
    with od.profile() as p:
        got = od.dion_rms_norm_backward(dy, h, rstd, w, dh=dh)
    torch.cuda.synchronize()
    assert (set(p.read()) == {"rms_norm_backward_small"}) == small
    check_backward(dy, h, rstd, w, dh, got, F32)
    own = dy.clone()
    with od.profile() as p:
        inplace = od.dion_rms_norm_backward(own, h, rstd, w, dh=dh, dx=own)
    torch.cuda.synchronize()
    assert "rms_norm_backward_small" not in p.read()
    check_backward(dy, h, rstd, w, dh, inplace, F32)


def test_backward_against_differences():
    """L = sum(dy * norm(h) w) + sum(dh * h): derivative along random directions, by
    central differences in 64 bits (error of order step^2) against the kernel's."""
    rows, cols, eps = 6, 200, 1e-6
    h, w, dy, dh = randn(rows, cols), 1 + 0.1 * randn(cols, seed=1), randn(rows, cols, seed=2), randn(rows, cols, seed=3)
    _, _, rstd = od.dion_rms_norm_q8(h, w, eps=eps)
    dx, dw = od.dion_rms_norm_backward(dy, h, rstd, w, dh=dh)
    H, W, DY, DH = (ref.f64(t) for t in (h, w, dy, dh))

    def loss(h_, w_):
        return (DY * ref.norm(h_, w_, eps)[0]).sum() + (DH * h_).sum()

    rng = np.random.default_rng(0)
    step = 1e-4
    for _ in range(5):
        u, v = rng.standard_normal(H.shape), rng.standard_normal(W.shape)
        for num, an, size in (((loss(H + step * u, W) - loss(H - step * u, W)) / (2 * step), (ref.f64(dx) * u).sum(),
                               np.abs(ref.f64(dx) * u).sum()),
                              ((loss(H, W + step * v) - loss(H, W - step * v)) / (2 * step), (ref.f64(dw) * v).sum(),
                               np.abs(ref.f64(dw) * v).sum())):
            assert abs(num - an) <= (TAU + 100 * step ** 2) * size


def test_backward_strides_in_place_and_empty():
    base = randn(4, 60, 270)
    w = 1 + 0.1 * randn(260, seed=1)
    rstd = torch.rand(60, device="cuda") + 0.5
    for off in (0, 3, 8):
        dy, h, dh = (base[i, :, off:off + 260] for i in range(3))
        check_backward(dy, h, rstd, w, dh, od.dion_rms_norm_backward(dy, h, rstd, w, dh=dh), F32)
        want = [t.clone() for t in od.dion_rms_norm_backward(dy, h, rstd, w, dh=dh)]
        for target in ("dy", "dh"):
            a, b = dy.clone(), dh.clone()
            got = od.dion_rms_norm_backward(a, h, rstd, w, dh=b, dx=a if target == "dy" else b)
            assert torch.allclose(got[0], want[0], rtol=1e-6, atol=1e-6) and torch.equal(got[1], want[1])
    e = torch.empty(0, 260, device="cuda")
    dx, dw = od.dion_rms_norm_backward(e, e, torch.empty(0, device="cuda"), w)
    assert dx.shape == (0, 260) and bool((dw == 0).all())


# ---------------------------------------------------- streams, graphs, refusals
def test_other_stream_and_graph():
    x, w = randn(200, 1024, dtype=BF16), torch.ones(1024, device="cuda")
    wt = randn(512, 1024, dtype=BF16, seed=1)
    w8, _ = od.dion_q8_quantize(wt, square=True)
    y0 = od.dion_q8_matmul(od.dion_rms_norm_q8(x, w)[0], w8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y1 = od.dion_q8_matmul(od.dion_rms_norm_q8(x, w, stream=s)[0], w8, stream=s)
    dx1 = od.dion_rms_norm_backward(x, x, torch.ones(200, device="cuda"), w, stream=s)
    s.synchronize()
    assert torch.equal(y0, y1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    xs = x.clone()
    with torch.cuda.graph(g):
        q, h, rstd = od.dion_rms_norm_q8(xs, w)
        y2 = od.dion_q8_matmul(q, w8)
        dx2 = od.dion_rms_norm_backward(xs, xs, rstd, w)
    for seed in (0, 9):
        xs.copy_(x if seed == 0 else randn(200, 1024, dtype=BF16, seed=seed))
        g.replay()
        q, _, rstd = od.dion_rms_norm_q8(xs, w)
        assert torch.equal(y2, od.dion_q8_matmul(q, w8))
        assert torch.equal(dx2[0], od.dion_rms_norm_backward(xs, xs, rstd, w)[0])
    assert dx1[0].shape == dx2[0].shape


def test_refusals():
    x, w = randn(4, 256), torch.ones(256, device="cuda")
    a = q8_operand(4, 256)
    with pytest.raises(ValueError, match="contiguous rows"):
        od.dion_q8_quantize(x.t())
    with pytest.raises(ValueError, match="overlapping"):
        od.dion_q8_quantize(x[:1].expand(4, 256))
    with pytest.raises(ValueError, match="go together"):
        od.dion_q8_quantize(x, rstd=torch.ones(4, device="cuda"))
    with pytest.raises(ValueError, match="16-byte"):
        od.dion_q8_matmul(od.Q8(torch.zeros(4, 264, dtype=torch.uint8, device="cuda").view(E4M3)[:, :256], a.scale), a)
    with pytest.raises(ValueError, match="4-byte"):
        od.dion_q8_matmul(od.Q8(a.data, torch.zeros(4, 6, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)[:, :2]), a)
    with pytest.raises(ValueError, match="do not fit"):
        od.dion_q8_matmul(od.Q8(a.data, a.scale[:, :1]), a)
    with pytest.raises(TypeError, match="e8m0"):
        od.dion_q8_matmul(od.Q8(a.data, torch.ones(4, 2, device="cuda")), a)
    with pytest.raises(TypeError, match="8-bit format"):
        od.dion_q8_matmul(od.Q8(x, a.scale), a)
    with pytest.raises(ValueError, match="out must be"):
        od.dion_q8_matmul(a, a, out=torch.empty(4, 5, device="cuda"))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        od.dion_q8_matmul(a, a, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="shape and dtype"):
        od.dion_rms_norm_q8(x, w, residual=x[:2])
    with pytest.raises(ValueError, match="vector"):
        od.dion_rms_norm_q8(x, w[:100])
    with pytest.raises(ValueError, match="only with a residual"):
        od.dion_rms_norm_q8(x, w, h=x)
    with pytest.raises(od.DionError):
        od.dion_rms_norm_q8(x, w, eps=-1.0)
    with pytest.raises(od.DionError):
        od.dion_rms_norm_backward(x, x, torch.ones(4, device="cuda"), w,
                                  workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="shape and dtype"):
        od.dion_rms_norm_backward(x, x.bfloat16(), torch.ones(4, device="cuda"), w)
    with pytest.raises(TypeError, match="float32"):
        od.dion_rms_norm_backward(x, x, torch.ones(4, dtype=BF16, device="cuda"), w)
