"""What is measured of the operators beside the orthonormal step, and their plain forms.

The step takes weight matrices; AdamW takes what is left of a model, all
tensors in one call, and the 4-bit products serve what was trained:

  gradnorm   norm = sqrt(sum of g^2 over all tensors), and the factor
             min(1, max_norm / (norm + 1e-6)) that a step scales gradients by
  adamw      g' = f g, m = b1 m + (1 - b1) g', v = b2 v + (1 - b2) g'^2,
             p = (1 - lr wd) p - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps);
             states in float32, or in 8 bits with one float32 scale for each
             256 values, E4M3 of m and of r = sqrt(v) (scale amax / 448); r is
             rounded up or down by a hash of the step's seed and number, the
             tensor and the element, and only a zero becomes zero
  quantize   groups of w along a row: s = bf16(amax / 7), q = rint(w / s), held
             in 4 bits, and the values that these stand for
  matmul     y = x (q s)^T for a few rows of x, plain or in 8 bits

`run` computes them in elementary torch operations in 32 bits, or, with `own`
set, by the package's calls.  `exact` is the same mathematics in 64 bits.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4, "q8": 1}
MAX_NORM = 1.0
LR, BETA1, BETA2, EPS, DECAY, SEED = 1e-3, 0.9, 0.999, 1e-8, 0.1, 20
BLOCK = 256                       # values of an 8-bit state that share a scale


def listed():
    return [
        # clipping what the orthonormal step leaves of a GPT-small model: norm weights and biases, position embedding
        dict(name="gradnorm-small", op="gradnorm", tensors="768*50+2304*12+786432", dtype="f32"),
        # the gradients of one Llama-3-8B layer
        dict(name="gradnorm-layer", op="gradnorm", tensors="16777216*2+4194304*2+58720256*3+4096*2", dtype="bf16"),
        # AdamW on the norm weights of a Llama-3-8B model alone: many small tensors, one launch's latency
        dict(name="adamw-norms", op="adamw", tensors="4096*65", p="bf16", g="bf16", state=32, copy=False),
        # the rest of a GPT-small model in float32: embeddings, norm weights, biases
        dict(name="adamw-embedding-f32", op="adamw", tensors="38597376+786432+768*50+2304*12", p="f32", g="f32",
             state=32, copy=False),
        # a 32000 x 4096 embedding and head with float32 master weights, their bfloat16 copy written along
        dict(name="adamw-master-copy", op="adamw", tensors="131072000*2+4096*65", p="f32", g="bf16", state=32, copy=True),
        # the same with states in 8 bits and bfloat16 weights, and tensors that end inside blocks and vectors
        dict(name="adamw-8bit", op="adamw", tensors="131072000*2+1*3+17+255+257*2+1000003+4096*60", p="bf16", g="bf16",
             state=8, copy=False),
        # a Llama-3-8B up projection laid out for serving
        dict(name="q4-quantize-14336x4096", op="quantize", n=14336, k=4096, dtype="bf16", group=128),
        # a ragged float32 matrix in fine groups, the last one of each row short
        dict(name="q4-quantize-1021x1000", op="quantize", n=1021, k=1000, dtype="f32", group=32),
        # one token at decode through an attention projection
        dict(name="q4-matmul-1x4096x4096", op="matmul", m=1, n=4096, k=4096, x="bf16", out="bf16", group=128),
        # a few float32 rows, sizes that end inside every tile
        dict(name="q4-matmul-5x1111x1000-f32", op="matmul", m=5, n=1111, k=1000, x="f32", out="f32", group=32),
        # sixteen requests at decode, the norm's 8-bit rows through a down projection
        dict(name="q4-matmul-16x4096x14336-q8", op="matmul", m=16, n=4096, k=14336, x="q8", out="bf16", group=64),
        # one token through a Llama-3-405B up projection
        dict(name="q4-matmul-1x53248x16384", op="matmul", m=1, n=53248, k=16384, x="bf16", out="bf16", group=128),
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gradnorm", "adamw", "adamw", "quantize", "matmul", "matmul", "matmul"])
    if op in ("gradnorm", "adamw"):
        parts, left = [], 1 << 27
        for _ in range(rng.randint(1, 4)):
            n = _log(rng, 1, left)
            times = _log(rng, 1, min(100, left // n))
            left = max(1, left - n * times)
            parts.append("%d*%d" % (n, times))
        case = dict(op=op, tensors="+".join(parts))
        if op == "gradnorm":
            return dict(case, dtype=rng.choice(["bf16", "f32"]))
        p = rng.choice(["bf16", "f32"])
        return dict(case, p=p, g=rng.choice(["bf16", "f32"]), state=rng.choice([8, 32]), copy=p == "f32" and rng.random() < 0.5)
    n, k, group = _log(rng, 16, 65536), _log(rng, 16, 16384), rng.choice([32, 64, 128, 128])
    if rng.random() < 0.6:
        n, k = max(64, n // 64 * 64), max(64, k // 64 * 64)
    if op == "quantize":
        return dict(op=op, n=min(n, (1 << 27) // k), k=k, dtype=rng.choice(["bf16", "bf16", "f32"]), group=group)
    return dict(op=op, m=rng.choice([1, 1, 1, 2, 3, 4, 5, 8, 13, 16]), n=min(n, 53248 * 16384 // (16 * k)), k=k,
                x=rng.choice(["bf16", "bf16", "f32", "q8"]), out=rng.choice(["bf16", "bf16", "f32"]), group=group)


# ------------------------------------------------------------------ inputs
def _sizes(text):
    """"768*2+100" -> [768, 768, 100]."""
    out = []
    for part in text.split("+"):
        n, _, times = part.partition("*")
        out += [int(n)] * int(times or 1)
    return out


def _starts(sizes):
    """Where each tensor starts in one allocation, on boundaries of BLOCK values, and its end."""
    at = [0]
    for n in sizes:
        at.append(at[-1] + -(-n // BLOCK) * BLOCK)
    return at


def _normal(gen, n, std):
    return torch.randn(n, generator=gen, device="cuda").mul_(std)


def _real(sizes, starts):
    """Which values of the allocation belong to a tensor."""
    bounds = torch.tensor([x for s, n in zip(starts, sizes) for x in (s, s + n)], device="cuda")
    return torch.bucketize(torch.arange(starts[-1], device="cuda"), bounds, right=True) % 2 == 1


def _prepare_tensors(case, gen, state):
    """The tensors of a list are views of one allocation each for weights, gradients and states."""
    sizes = _sizes(case["tensors"])
    starts = _starts(sizes)
    total, real = starts[-1], _real(sizes, starts)
    views = lambda t: [t[s:s + n] for s, n in zip(starts, sizes)]  # noqa: E731
    state["starts"] = torch.tensor(starts[:-1], device="cuda")
    # each tensor's gradients have a magnitude of their own, and heavier tails than a normal's
    spread = torch.exp(_normal(gen, total // BLOCK, 1.0)).repeat_interleave(BLOCK)
    grad = _normal(gen, total, 1e-3).mul_(spread).mul_(real)
    if case["op"] == "gradnorm":
        state["g"] = grad.to(TYPES[case["dtype"]])
        if own:
            import orthonormal_optimizer_step_gb300 as od
            state["list"] = od.dion_grad_list(views(state["g"]))
        return
    state["g"] = grad.to(TYPES[case["g"]])
    state["p"] = _normal(gen, total, 0.02).mul_(real).to(TYPES[case["p"]])
    state["copy"] = torch.zeros(total, dtype=torch.bfloat16, device="cuda") if case["copy"] else None
    m = _normal(gen, total, 3e-4).mul_(spread).mul_(real)
    v = (_normal(gen, total, 1e-3).mul_(spread).square_().add_(1e-9)).mul_(real)
    if case["state"] == 8:
        state["m"], state["ms"] = _m_codes(m)
        state["r"], state["rs"] = _r_codes(v.sqrt(), torch.full((total,), 1 << 19, device="cuda"))
    else:
        state["m"], state["v"] = m, v
    state["step"] = 1000
    # the norm's second value: a device scalar that the step reads
    state["factor"] = torch.full((1,), 0.7, device="cuda")
    if own:
        import orthonormal_optimizer_step_gb300 as od
        if case["state"] == 8:
            blocks = lambda t: [t[s // BLOCK:(s + n + BLOCK - 1) // BLOCK] for s, n in zip(starts, sizes)]  # noqa: E731
            first = [od.State8(*x) for x in zip(views(state["m"]), blocks(state["ms"]))]
            second = [od.State8(*x) for x in zip(views(state["r"]), blocks(state["rs"]))]
        else:
            first, second = views(state["m"]), views(state["v"])
        state["plan"] = od.dion_adamw_plan(views(state["p"]), views(state["g"]), first, second,
                                           copies=views(state["copy"]) if case["copy"] else None)


def _chunks(k):
    return -(-k // 128)


def _pack(q):
    """Whole numbers -8..7 [n, k] -> the held 4-bit rows: 64 bytes for each 128 columns, 32-bit word 4 t + j of them
    with columns 32 j + 8 t + (0, 2, 4, 6, 1, 3, 5, 7) from its low end, each plus eight; columns past k hold zero."""
    n, k = q.shape
    full = torch.zeros(n, _chunks(k) * 128, dtype=torch.int64, device=q.device)
    full[:, :k] = q
    c = (full + 8).view(n, _chunks(k), 4, 4, 4, 2).permute(0, 1, 3, 2, 5, 4).reshape(n, _chunks(k) * 16, 8)
    word = (c << (4 * torch.arange(8, device=q.device))).sum(-1)
    return ((word + (1 << 31)) % (1 << 32) - (1 << 31)).to(torch.int32).view(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = dict(case)
    if case["op"] in ("gradnorm", "adamw"):
        _prepare_tensors(case, gen, state)
        return state
    n, k = case["n"], case["k"]
    w = torch.randn(n, k, generator=gen, device="cuda").mul_(0.02)
    if case["op"] == "quantize":
        state["w"] = w.to(TYPES[case["dtype"]])
        return state
    q, s = _groups(w.to(torch.bfloat16).float(), case["group"])
    state["q"], state["s"] = torch.cat([_pack(x) for x in q.split(4096)]), s
    # activations: each column has a magnitude of its own
    x = torch.randn(case["m"], k, generator=gen, device="cuda") * torch.exp(0.5 * torch.randn(k, generator=gen, device="cuda"))
    if case["x"] == "q8":
        # as the norm leaves them: E4M3 in blocks of 128 with power-of-two scales, rows on 16-byte boundaries
        xb = torch.zeros(case["m"], _chunks(k) * 128, device="cuda")
        xb[:, :k] = x
        xb = xb.view(case["m"], -1, 128)
        ex = torch.ceil(torch.log2(xb.abs().amax(-1) / 448.0)).clamp(-126, 126)
        q8 = (xb * torch.exp2(-ex).unsqueeze(-1)).to(torch.float8_e4m3fn).view(case["m"], -1)
        scale = torch.zeros(case["m"], -(-_chunks(k) // 4) * 4, dtype=torch.uint8, device="cuda")
        scale[:, :_chunks(k)] = (ex + 127).to(torch.uint8)
        state["x8"], state["xs"] = q8[:, :k], scale.view(torch.float8_e8m0fnu)[:, :_chunks(k)]
    else:
        state["x8"], state["xs"] = x.to(TYPES[case["x"]]), None
    return state


# ------------------------------------------------------------- plain forms
def _m_codes(m):
    """float32 -> E4M3 values and the scales of their blocks."""
    blocks = m.view(-1, BLOCK)
    amax = blocks.abs().amax(-1)
    scale = (amax / torch.full_like(amax, 448.0)).clamp(min=2.0 ** -100)
    return (blocks * (1.0 / scale).unsqueeze(-1)).to(torch.float8_e4m3fn).view(-1), scale


def _r_codes(r, dither):
    """float32 >= 0 -> E4M3 values, rounded up where 20 bits of dither carry, and the scales of their blocks."""
    blocks = r.view(-1, BLOCK)
    rmax = blocks.amax(-1)
    scale = (rmax / torch.full_like(rmax, 448.0)).clamp(min=2.0 ** -100)
    # times 2^-120 a float's exponent is that of E4M3, subnormals included, and its top 3 mantissa bits are E4M3's
    x = (blocks * (1.0 / scale).unsqueeze(-1)).view(-1) * 2.0 ** -120
    code = (x.view(torch.int32) + dither.to(torch.int32)) >> 20
    return torch.where(r > 0, code.clamp(1, 126), torch.zeros_like(code)).to(torch.uint8).view(torch.float8_e4m3fn), scale


def _mix(x):
    """A hash of 32-bit numbers held in 64: two rounds of shift, exclusive or and product."""
    x = ((x ^ (x >> 16)) * 0x9E3779B1) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x85EBCA6B) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _dither(starts, total, step):
    """20 bits for each value of the allocation, from the seed, the step, the tensor and the place in it."""
    key = _mix(torch.tensor([(SEED * 0x632BE5AB + step) & 0xFFFFFFFF], device=starts.device))
    keys = _mix(key ^ torch.arange(len(starts), device=starts.device))
    at = torch.arange(total, device=starts.device)
    tensor = torch.bucketize(at, starts, right=True) - 1
    return _mix((at - starts[tensor]) ^ keys[tensor]) >> 12


def _groups(w, group):
    """float32 [n, k] -> whole numbers -8..7 (int8) and the bfloat16 scales of groups along the rows."""
    n, k = w.shape
    g = -(-k // group)
    full = torch.zeros(n, g * group, device=w.device)
    full[:, :k] = w
    full = full.view(n, g, group)
    amax = full.abs().amax(-1)
    s = (amax / torch.full_like(amax, 7.0)).to(torch.bfloat16)
    # (a quotient that is half-way between two is rounded to the even one, so it has to be a division)
    by = torch.where(s > 0, s.float(), torch.ones_like(amax))
    return torch.round(full / by.unsqueeze(-1)).clamp(-8, 7).to(torch.int8).view(n, -1)[:, :k], s


def _unpack(q, k):
    """The held 4-bit rows -> float32 whole numbers [n, k]."""
    n = q.shape[0]
    word = q.view(torch.int32).view(n, -1, 4, 4, 1, 1)
    shift = (4 * torch.arange(8, device=q.device, dtype=torch.int32)).view(2, 4)
    c = (word >> shift) & 15                                       # [n, chunk, t, j, odd, pair]
    return c.permute(0, 1, 3, 2, 5, 4).reshape(n, -1)[:, :k].float() - 8.0


def _plain_adamw(st):
    st["step"] += 1
    g = st["g"].float() * st["factor"]
    if st["state"] == 8:
        m = (st["m"].float().view(-1, BLOCK) * st["ms"].unsqueeze(-1)).view(-1)
        v = (st["r"].float().view(-1, BLOCK) * st["rs"].unsqueeze(-1)).view(-1).square()
    else:
        m, v = st["m"], st["v"]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    root = v.sqrt()
    p = st["p"].float() * (1 - LR * DECAY)
    p = p - m * (LR / (1 - BETA1 ** st["step"])) / (root * (1 / math.sqrt(1 - BETA2 ** st["step"])) + EPS)
    st["p"].copy_(p)
    if st["copy"] is not None:
        st["copy"].copy_(p)
    if st["state"] == 8:
        for name, t in zip(("m", "ms", "r", "rs"), _m_codes(m) + _r_codes(root, _dither(st["starts"], len(p), st["step"]))):
            st[name].copy_(t)
    else:
        st["m"].copy_(m)
        st["v"].copy_(v)
    return _stepped(st)


def _stepped(st):
    names = ("p", "copy", "m", "ms", "r", "rs") if st["state"] == 8 else ("p", "copy", "m", "v")
    return {name: st[name] for name in names}


def _x_values(st):
    if st["xs"] is None:
        return st["x8"].float()
    ex = st["xs"].view(torch.uint8).to(torch.int32) << 23
    return st["x8"].float() * ex.view(torch.float32).repeat_interleave(128, 1)[:, :st["k"]]


def _plain(st):
    op = st["op"]
    if op == "gradnorm":
        # (long sums: in 64 bits)
        norm = st["g"].float().square().sum(dtype=torch.float64).sqrt()
        return {"norm": torch.stack([norm, (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)]).float()}
    if op == "adamw":
        return _plain_adamw(st)
    if op == "quantize":
        q, s = _groups(st["w"].float(), st["group"])
        values = _unpack(_pack(q), st["k"]) * s.float().repeat_interleave(st["group"], 1)[:, :st["k"]]
        return {"w": values.to(TYPES[st["dtype"]]), "s": s}
    w = _unpack(st["q"], st["k"]) * st["s"].float().repeat_interleave(st["group"], 1)[:, :st["k"]]
    return {"y": (_x_values(st) @ w.t()).to(TYPES[st["out"]])}


# ------------------------------------------------------- the package's calls
def _own(st):
    import orthonormal_optimizer_step_gb300 as od

    op = st["op"]
    if op == "gradnorm":
        return {"norm": od.dion_grad_norm(st["list"], max_norm=MAX_NORM)}
    if op == "adamw":
        st["step"] += 1
        od.dion_adamw_step(st["plan"], step=st["step"], lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY,
                           grad_scale=st["factor"], seed=SEED)
        return _stepped(st)
    if op == "quantize":
        w = od.dion_q4_quantize(st["w"], group=st["group"])
        return {"w": od.dion_q4_dequantize(w, out_dtype=TYPES[st["dtype"]]), "s": w.scale}
    x = st["x8"] if st["xs"] is None else od.Q8(st["x8"], st["xs"])
    return {"y": od.dion_q4_matmul(x, od.Q4(st["q"], st["s"], st["k"], st["group"]), out_dtype=TYPES[st["out"]])}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op in ("gradnorm", "adamw"):
        n = sum(_sizes(case["tensors"]))
        if op == "gradnorm":
            return {"bytes": n * BYTES[case["dtype"]] + 8, "flops": 2 * n}
        blocks = sum(-(-x // BLOCK) for x in _sizes(case["tensors"]))
        states = 4 * n + 16 * blocks if case["state"] == 8 else 16 * n
        return {"bytes": n * (2 * BYTES[case["p"]] + BYTES[case["g"]] + (2 if case["copy"] else 0)) + states, "flops": 15 * n}
    n, k, groups = case["n"], case["k"], -(-case["k"] // case["group"])
    held = n * (_chunks(k) * 64 + 2 * groups)
    if op == "quantize":
        return {"bytes": 2 * n * k * BYTES[case["dtype"]] + held, "flops": 4 * n * k}
    m = case["m"]
    scales = m * _chunks(k) if case["x"] == "q8" else 0
    return {"bytes": held + m * k * BYTES[case["x"]] + scales + m * n * BYTES[case["out"]], "flops": 2 * m * n * k}


# ------------------------------------------------------------------- 64 bits
def _step_of(x, bits, low):
    """The distance between neighbouring values of a float format at x >= 0 (float64): bits of mantissa, least exponent."""
    _, ex = torch.frexp(x)
    return (((ex - 1).clamp(min=low) - bits + 1023).to(torch.int64) << 52).view(torch.float64)   # exact, as a library's power is not


def _exact_hash(x):
    x = ((x ^ x // 65536) * 2654435761) % 4294967296
    x = ((x ^ x // 32768) * 2246822507) % 4294967296
    return x ^ x // 65536


def _exact_dither(sizes, total, step):
    """In [0, 1): the value's share of a step that it may be rounded up by."""
    out = torch.zeros(total, dtype=torch.float64, device="cuda")
    key = _exact_hash(torch.tensor((SEED * 0x632BE5AB + step) % 4294967296, device="cuda"))
    for i, (s, n) in enumerate(zip(_starts(sizes), sizes)):
        out[s:s + n] = (_exact_hash(torch.arange(n, device="cuda") ^ _exact_hash(key ^ i)) // 4096).double() / 2 ** 20
    return out


def _exact_adamw(case, st):
    t = st["step"] + 1
    f, p = st["factor"].double(), st["p"].double()
    g = st["g"].double() * f
    if case["state"] == 8:
        m = (st["m"].double().view(-1, BLOCK) * st["ms"].double()[:, None]).flatten()
        v = ((st["r"].double().view(-1, BLOCK) * st["rs"].double()[:, None]) ** 2).flatten()
    else:
        m, v = st["m"].double(), st["v"].double()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g ** 2
    update = (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS)
    p = p - LR * (update + DECAY * p)
    out = {"p": p, "copy": p if case["copy"] else None}
    if case["state"] == 32:
        return {**out, "m": m, "v": v}
    ms = (m.abs().view(-1, BLOCK).amax(1) / 448).clamp(min=2.0 ** -100)
    x = (m.view(-1, BLOCK) / ms[:, None]).flatten()
    step = _step_of(x.abs(), 3, -6)
    r = torch.sqrt(v)
    rs = (r.view(-1, BLOCK).amax(1) / 448).clamp(min=2.0 ** -100)
    y = (r.view(-1, BLOCK) / rs[:, None]).flatten()
    up = _step_of(y, 3, -6)
    y = (torch.floor(y / up + _exact_dither(_sizes(case["tensors"]), len(p), t)) * up).clamp(2.0 ** -9, 448)
    return {**out, "m": torch.round(x / step) * step, "ms": ms, "r": torch.where(r > 0, y, 0.0), "rs": rs}


def _exact_values(q, s, k, group):
    """Held 4-bit rows -> their values, column by column of the layout."""
    nibble = torch.stack([q & 15, q >> 4], -1).view(q.shape[0], -1)            # in the order of the bits
    col = torch.arange(k, device=q.device)
    c = col % 128
    j, t, e = c // 32, c % 32 // 8, c % 8
    at = col // 128 * 128 + (4 * t + j) * 8 + e // 2 + 4 * (e % 2)
    return (nibble[:, at].double() - 8) * s.double()[:, col // group]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "gradnorm":
        norm = torch.linalg.vector_norm(st["g"].double())
        return {"norm": torch.stack([norm, (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)])}
    if op == "adamw":
        return _exact_adamw(case, st)
    k, group = case["k"], case["group"]
    if op == "quantize":
        w, s, out = st["w"].double(), [], torch.zeros_like(st["w"], dtype=torch.float64)
        for c in range(0, k, group):
            part = w[:, c:c + group]
            amax = part.abs().amax(1, keepdim=True)
            unit = _step_of(amax / 7, 7, -126)
            scale = torch.round(amax / 7 / unit) * unit
            out[:, c:c + group] = torch.where(scale > 0, (part / scale).round().clamp(-8, 7) * scale, 0.0)
            s.append(scale)
        return {"w": out, "s": torch.cat(s, 1)}
    x = st["x8"].double()
    if st["xs"] is not None:
        x = x * torch.exp2(st["xs"].view(torch.uint8).double() - 127)[:, torch.arange(k, device="cuda") // 128]
    rows = [torch.einsum("mk,nk->mn", x, _exact_values(q, s, k, group)) for q, s in zip(st["q"].split(4096), st["s"].split(4096))]
    return {"y": torch.cat(rows, 1)}
