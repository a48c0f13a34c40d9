"""What is measured of the 8-bit linear layer's operators, and their plain forms.

A linear layer whose weights the orthonormal step trains reads its activations,
weights and gradients in 8-bit floating point, each block of 128 values along
the contraction with a power-of-two scale:

  quantize       x -> q, s: q = round8(x / s), s = 2^e the smallest power of two
                 with max|x| <= 448 s over the block (57344 s for e5m2); blocks
                 are 1 x 128 along a row, 128 x 1 down a column (the transposed
                 copy) or 128 x 128 (weights, both orders from one scale)
  matmul         C = (qa sa) (qb sb)^T, both operands contracted along their rows
  norm           h = x + residual, y = h / sqrt(mean(h^2) + eps) * w, and y's q, s
  norm_backward  from dy: dx = rstd (w dy - xhat mean(w dy xhat)) + dh and
                 dw = sum over the rows of dy xhat, xhat = h rstd

`run` computes them in elementary torch operations in 32 bits, or, with `own`
set, by the package's calls.  `exact` is the same mathematics in 64 bits with
no intermediate rounding.
"""
import math

import torch

own = False

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": E4M3, "e5m2": E5M2}
BYTES = {"bf16": 2, "f32": 4}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
EPS = 1e-6


def listed():
    return [
        # one token at decode: the residual's addition and the norm before a Llama-3-8B projection
        dict(name="norm-1x4096", op="norm", rows=1, cols=4096, dtype="bf16", residual=True),
        # a training micro-batch of 8192 tokens at the same width
        dict(name="norm-8192x4096", op="norm", rows=8192, cols=4096, dtype="bf16", residual=True),
        # a ragged batch in float32, last block of each row short, no residual
        dict(name="norm-1021x1000-f32", op="norm", rows=1021, cols=1000, dtype="f32", residual=False),
        # the norm's gradient for a short GPT-small sequence
        dict(name="normbwd-100x768", op="norm_backward", rows=100, cols=768, dtype="bf16", residual=True),
        # and for the 8192-token micro-batch, with the residual stream's own gradient added
        dict(name="normbwd-8192x4096", op="norm_backward", rows=8192, cols=4096, dtype="bf16", residual=True),
        # GPT-small's attention projections after the optimizer step: both orders of 12 matrices
        dict(name="quant-weights-12x768x2304", op="quantize", batch=12, rows=768, cols=2304, dtype="bf16",
             format="e4m3", form="both", square=True),
        # an output gradient in training: rows for dX, columns for dW; the wider-range format
        dict(name="quant-grad-8192x4096", op="quantize", batch=1, rows=8192, cols=4096, dtype="bf16",
             format="e5m2", form="both", square=False),
        # one token at decode through a Llama-3-8B up projection
        dict(name="matmul-1x14336x4096", op="matmul", m=1, n=14336, k=4096, out="bf16", a_format="e4m3",
             b_square=True),
        # a few tokens in flight, sizes that end inside every tile and block
        dict(name="matmul-37x1111x1000", op="matmul", m=37, n=1111, k=1000, out="f32", a_format="e4m3",
             b_square=True),
        # a short GPT-small batch through its attention projections
        dict(name="matmul-1024x2304x768", op="matmul", m=1024, n=2304, k=768, out="bf16", a_format="e4m3",
             b_square=True),
        # the training forward of the up projection
        dict(name="matmul-8192x14336x4096", op="matmul", m=8192, n=14336, k=4096, out="bf16", a_format="e4m3",
             b_square=True),
        # a weight gradient for the optimizer: contracted over the tokens, scales down the columns of both
        dict(name="matmul-dw-4096x4096x8192", op="matmul", m=4096, n=4096, k=8192, out="bf16", a_format="e5m2",
             b_square=False),
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "quantize", "matmul", "matmul"])
    if op in ("norm", "norm_backward"):
        cols = _log(rng, 64, 16384)
        if rng.random() < 0.5:
            cols = max(64, cols // 64 * 64)
        return dict(op=op, rows=_log(rng, 1, min(16384, (1 << 25) // cols)), cols=cols,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), residual=rng.random() < 0.7)
    if op == "quantize":
        batch = rng.choice([1, 1, 2, 12])
        cols = _log(rng, 48, 16384)
        if rng.random() < 0.5:
            cols = max(64, cols // 64 * 64)
        return dict(op=op, batch=batch, rows=_log(rng, 1, min(16384, (1 << 25) // (cols * batch))), cols=cols,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), format=rng.choice(["e4m3", "e4m3", "e5m2"]),
                    form=rng.choice(["rows", "cols", "both"]), square=rng.random() < 0.4)
    n, k = _log(rng, 64, 14336), _log(rng, 64, 14336)
    if rng.random() < 0.6:
        n, k = max(64, n // 64 * 64), max(64, k // 64 * 64)
    most = 8192 * 14336 * 4096 // (n * k)
    return dict(op=op, m=_log(rng, 1, max(1, min(16384, most))), n=n, k=k, out=rng.choice(["bf16", "bf16", "f32"]),
                a_format=rng.choice(["e4m3", "e4m3", "e5m2"]), b_square=rng.random() < 0.6)


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, std, dtype, spread=0.0):
    """N(0, std^2); with `spread`, each column has a magnitude of its own, as activations do."""
    t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    t.mul_(std)
    if spread:
        t.mul_(torch.exp(spread * torch.randn(shape[-1], generator=gen, device="cuda")))
    return t.to(dtype)


def _held(q, s):
    """The 8-bit matrix as a program keeps it: rows start on 16-byte, scale rows on 4-byte boundaries."""
    (r, c), (sr, sc) = q.shape, s.shape
    data = torch.zeros(r, (c + 15) // 16 * 16, dtype=torch.uint8, device="cuda").view(q.dtype)[:, :c]
    scale = torch.zeros(sr, (sc + 3) // 4 * 4, dtype=torch.uint8, device="cuda").view(s.dtype)[:, :sc]
    data.view(torch.uint8).copy_(q.view(torch.uint8))
    scale.view(torch.uint8).copy_(s.view(torch.uint8))
    return data, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = dict(case)
    op = case["op"]
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        x = _normal(gen, (m, k), 1.0, torch.bfloat16, 0.5)
        w = _normal(gen, (n, k), 0.02, torch.bfloat16)
        state["a"] = _held(*_blocks(x.float(), case["a_format"], False))
        state["b"] = _held(*_blocks(w.float(), "e4m3", case["b_square"]))
        return state
    dt = TYPES[case["dtype"]]
    if op == "quantize":
        shape = (case["batch"], case["rows"], case["cols"])
        state["x"] = _normal(gen, shape, 0.02, dt) if case["square"] else _normal(gen, shape, 1e-3, dt, 1.0)
        return state
    shape = (case["rows"], case["cols"])
    state["w"] = (1.0 + 0.1 * torch.randn(shape[1], generator=gen, device="cuda")).to(dt)
    state["x"] = _normal(gen, shape, 1.0, dt, 0.5)
    state["r"] = _normal(gen, shape, 2.0, dt, 0.5) if case["residual"] else None
    if op == "norm_backward":
        h = state["x"]
        state["rstd"] = 1.0 / torch.sqrt(h.float().square().mean(-1) + EPS)
        state["dy"] = _normal(gen, shape, 1e-2, dt)
        state["r"] = _normal(gen, shape, 1e-2, dt) if case["residual"] else None
    return state


# ------------------------------------------------------------- plain forms
def _cut(x):
    """[..., r, c] -> [..., r, blocks, 128], the last block filled with zeros."""
    c = x.shape[-1]
    pad = -c % 128
    if pad:
        x = torch.cat([x, x.new_zeros(x.shape[:-1] + (pad,))], -1)
    return x.view(x.shape[:-1] + ((c + pad) // 128, 128))


def _amax_square(amax):
    """Maxima of 1 x 128 blocks -> of 128 x 128 blocks."""
    r = amax.shape[-2]
    pad = -r % 128
    if pad:
        amax = torch.cat([amax, amax.new_zeros(amax.shape[:-2] + (pad, amax.shape[-1]))], -2)
    return amax.view(amax.shape[:-2] + ((r + pad) // 128, 128, amax.shape[-1])).amax(-2)


def _power(ex):
    """2^ex in float32, exact for whole -252 <= ex <= 254 (a library power may be off in its last bit)."""
    half = ex.to(torch.int32) // 2
    return ((half + 127) << 23).view(torch.float32) * ((ex.to(torch.int32) - half + 127) << 23).view(torch.float32)


def _blocks(x, fmt, square):
    """float32 [..., r, c] -> 8-bit values and scales of its blocks along the rows."""
    xb = _cut(x)
    amax = xb.abs().amax(-1)
    if square:
        amax = _amax_square(amax)
    mant, ex = torch.frexp(amax / LARGEST[fmt])
    ex = torch.where(mant == 0.5, ex - 1, ex).clamp(-127, 127)
    ex = torch.where(amax == 0, torch.zeros_like(ex), ex)
    down = _power(-ex)
    if square:
        down = down.repeat_interleave(128, -2)[..., :x.shape[-2], :]
    q = (xb * down.unsqueeze(-1)).flatten(-2)[..., :x.shape[-1]]
    return q.to(TYPES[fmt]), (ex + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _values(q, s, rows):
    """8-bit values and scales -> float32."""
    ex = _power(s.view(torch.uint8).to(torch.int32) - 127)
    if ex.shape[0] != rows:
        ex = ex.repeat_interleave(128, 0)[:rows]
    return (_cut(q.float()) * ex.unsqueeze(-1)).flatten(-2)[:, :q.shape[1]]


def _plain(st):
    op = st["op"]
    if op == "matmul":
        a, b = _values(*st["a"], st["m"]), _values(*st["b"], st["n"])
        return {"c": (a @ b.t()).to(TYPES[st["out"]])}
    if op == "quantize":
        x, out = st["x"].float(), {}
        if st["form"] in ("rows", "both"):
            out["q"], out["s"] = _blocks(x, st["format"], st["square"])
        if st["form"] in ("cols", "both"):
            out["qt"], out["st"] = _blocks(x.transpose(-2, -1).contiguous(), st["format"], st["square"])
        return out
    x, w = st["x"], st["w"].float()
    if op == "norm":
        h = x if st["r"] is None else (x.float() + st["r"].float()).to(x.dtype)
        f = h.float()
        rstd = 1.0 / torch.sqrt(f.square().mean(-1) + EPS)
        q, s = _blocks(f * rstd.unsqueeze(-1) * w, "e4m3", False)
        return {"h": h, "q": q, "s": s, "rstd": rstd}
    xhat = x.float() * st["rstd"].unsqueeze(-1)
    dy = st["dy"].float()
    g = dy * w
    dx = (g - xhat * (g * xhat).mean(-1, keepdim=True)) * st["rstd"].unsqueeze(-1)
    if st["r"] is not None:
        dx = dx + st["r"].float()
    return {"dx": dx.to(x.dtype), "dw": (dy * xhat).sum(0)}


# ------------------------------------------------------- the package's calls
def _own(st):
    import orthonormal_optimizer_step_gb300 as od

    op = st["op"]
    if op == "matmul":
        return {"c": od.dion_q8_matmul(od.Q8(*st["a"]), od.Q8(*st["b"]), out_dtype=TYPES[st["out"]])}
    if op == "quantize":
        rows, cols = od.dion_q8_quantize(st["x"], form=st["form"], square=st["square"], dtype=TYPES[st["format"]])
        out = {}
        if rows is not None:
            out["q"], out["s"] = rows
        if cols is not None:
            out["qt"], out["st"] = cols
        return out
    if op == "norm":
        y, h, rstd = od.dion_rms_norm_q8(st["x"], st["w"], residual=st["r"], eps=EPS)
        return {"h": h, "q": y.data, "s": y.scale, "rstd": rstd}
    dx, dw = od.dion_rms_norm_backward(st["dy"], st["x"], st["rstd"], st["w"], dh=st["r"])
    return {"dx": dx, "dw": dw}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // 128)
        scales = kb * (m + (-(-n // 128) if case["b_square"] else n))
        return {"bytes": m * k + n * k + scales + m * n * BYTES[case["out"]], "flops": 2 * m * n * k}
    r, c, e = case["rows"], case["cols"], BYTES[case["dtype"]]
    if op == "quantize":
        orders = 2 if case["form"] == "both" else 1
        one = r * c * (e + orders)
        rb, cb = -(-r // 128), -(-c // 128)
        if case["form"] in ("rows", "both"):
            one += cb * (rb if case["square"] else r)
        if case["form"] in ("cols", "both"):
            one += rb * (cb if case["square"] else c)
        return {"bytes": case["batch"] * one, "flops": case["batch"] * r * c * (1 + orders)}
    if op == "norm":
        moved = r * c * (e + 1 + (2 * e if case["residual"] else 0)) + r * (-(-c // 128)) + 4 * r + c * e
        return {"bytes": moved, "flops": 6 * r * c}
    moved = r * c * (3 * e + (e if case["residual"] else 0)) + 4 * r + c * (e + 4)
    return {"bytes": moved, "flops": 10 * r * c}


# ------------------------------------------------------------------- 64 bits
def _power64(ex):
    """2^ex in float64 for whole |ex| < 1000, from the exponent's bits."""
    return ((ex.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round8(v, fmt):
    """float64 -> nearest value of the 8-bit format, ties to even."""
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    _, ex = torch.frexp(v)
    step = _power64((ex - 1).clamp(min=low) - bits)
    return torch.round(v / step) * step


def _exact_blocks(x, fmt, square):
    r, c = x.shape[-2:]
    rb, cb = -(-r // 128), -(-c // 128)
    full = torch.zeros(x.shape[:-2] + (rb * 128, cb * 128), dtype=torch.float64, device=x.device)
    full[..., :r, :c] = x
    tiles = full.view(x.shape[:-2] + (rb, 128, cb, 128))
    top = tiles.abs().amax((-3, -1) if square else -1, keepdim=True)
    ex = torch.ceil(torch.log2(top.clamp(min=1e-300) / LARGEST[fmt]))   # rounded: mended by one either way
    ex = torch.where(LARGEST[fmt] * _power64(ex - 1) >= top, ex - 1, ex)
    ex = torch.where(LARGEST[fmt] * _power64(ex) < top, ex + 1, ex)
    ex = torch.where(top > 0, ex.clamp(-127, 127), torch.zeros_like(ex))
    s = _power64(ex)
    q = _round8(tiles / s, fmt).view(full.shape)[..., :r, :c]
    s = s.squeeze(-1)
    s = s.squeeze(-2) if square else s.flatten(-3, -2)[..., :r, :]
    return q, s


def _exact_values(q, s, rows):
    q = q.double()
    step = _power64(s.view(torch.uint8).long() - 127)
    row = torch.arange(rows, device=q.device)
    if step.shape[0] != rows:
        row = row // 128
    col = torch.arange(q.shape[1], device=q.device) // 128
    return q * step[row][:, col]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "matmul":
        return {"c": torch.einsum("mk,nk->mn", _exact_values(*st["a"], case["m"]), _exact_values(*st["b"], case["n"]))}
    x = st["x"].double()
    if op == "quantize":
        out = {}
        if case["form"] != "cols":
            out["q"], out["s"] = _exact_blocks(x, case["format"], case["square"])
        if case["form"] != "rows":
            out["qt"], out["st"] = _exact_blocks(x.mT, case["format"], case["square"])
        return out
    w = st["w"].double()
    if op == "norm":
        h = x + st["r"].double() if case["residual"] else x
        rstd = torch.rsqrt((h * h).sum(1) / case["cols"] + EPS)
        q, s = _exact_blocks(h * rstd[:, None] * w, "e4m3", False)
        return {"h": h, "q": q, "s": s, "rstd": rstd}
    rstd, dy = st["rstd"].double()[:, None], st["dy"].double()
    xhat = x * rstd
    mean = (dy * w * xhat).sum(1, keepdim=True) / case["cols"]
    dx = rstd * (dy * w - xhat * mean)
    if case["residual"]:
        dx = dx + st["r"].double()
    return {"dx": dx, "dw": torch.einsum("tc,tc->c", dy, xhat)}
