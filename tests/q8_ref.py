"""Plain 64-bit implementations of the 8-bit linear layer's operators, in numpy."""
import numpy as np
import torch

FORMATS = {torch.float8_e4m3fn: (448.0, 3, -6), torch.float8_e5m2: (57344.0, 2, -14)}


def f64(t):
    return t.detach().to(torch.float32).to(torch.float64).cpu().numpy()


def round8(v, dtype):
    """Nearest value of the format, ties to even (no overflow: |v| <= the largest value)."""
    _, bits, low = FORMATS[dtype]
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e - 1, low) - bits)
    return np.rint(v / step) * step


def block_exponents(x, dtype, square):
    """Exponents of the blocks' scales; only finite values count."""
    top = FORMATS[dtype][0]
    r, c = x.shape
    kb = -(-c // 128)
    mag = np.zeros((r, kb * 128))
    mag[:, :c] = np.where(np.isfinite(x), np.abs(x), 0.0)
    a = mag.reshape(r, kb, 128).max(-1)
    if square:
        pad = np.zeros((-(-r // 128) * 128, kb))
        pad[:r] = a
        a = pad.reshape(-1, 128, kb).max(1)
    m, e = np.frexp(a / top)                       # exact: top is 1.75 times a power of two, a has 24 bits
    e = np.where(a > top * np.ldexp(1.0, np.where(m == 0.5, e - 1, e)), e + 1, np.where(m == 0.5, e - 1, e))
    return np.where(a > 0, np.maximum(e, -127), 0)


def spread(e, rows, cols):
    """Block scales' exponents -> one for each element."""
    if e.shape[0] != rows:
        e = np.repeat(e, 128, 0)[:rows]
    return np.repeat(e, 128, 1)[:, :cols]


def quantize(x, dtype, square=False):
    e = block_exponents(x, dtype, square)
    with np.errstate(invalid="ignore"):
        v = np.ldexp(x, -spread(e, *x.shape))
        return np.where(np.isfinite(x), round8(np.where(np.isfinite(x), v, 0.0), dtype), np.nan), e


def exponents(scale):
    return scale.view(torch.uint8).cpu().numpy().astype(np.int64) - 127


def values(q):
    """Q8 -> float64 values."""
    return np.ldexp(f64(q.data), spread(exponents(q.scale), *q.data.shape))


def norm(h, w, eps):
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * w, rstd


def norm_backward(dy, h, rstd, w, dh=None):
    xhat = h * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - xhat * (g * xhat).mean(1, keepdims=True))
    return dx + (0.0 if dh is None else dh), (dy * xhat).sum(0)
