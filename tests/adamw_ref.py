"""AdamW and the rounding of its 8-bit states in float64, one tensor at a time."""
import math

import numpy as np
import torch

BLOCK = 256


def values(state, n):
    """float64 values of a State8 of n elements."""
    s = state.scale.double().repeat_interleave(BLOCK)[:n]
    return state.data.flatten().double() * s


def step(p, g, m, v, t, *, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, scale=1.0):
    """(p, m, v) after the step and the size of p's update and of its terms, all float64."""
    g = g.double() * scale
    m1 = betas[0] * m + (1 - betas[0]) * g
    v1 = betas[1] * v + (1 - betas[1]) * g * g
    rate = lr / (1 - betas[0] ** t)
    root = torch.sqrt(v1 / (1 - betas[1] ** t)) + eps
    size = rate * (betas[0] * m.abs() + (1 - betas[0]) * g.abs()) / root
    return p.double() * (1 - lr * weight_decay) - rate * m1 / root, m1, v1, size


def mix(x):
    x = np.uint64(x) & np.uint64(0xFFFFFFFF)
    m = np.uint64(0xFFFFFFFF)
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x9E3779B1)) & m
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0x85EBCA6B)) & m
    return x ^ (x >> np.uint64(16))


def dither(n, seed, t, index, start=0):
    """In [0, 1), for elements start .. start + n - 1 of the list's tensor `index`."""
    key = mix((seed * 0x632BE5AB + t) & 0xFFFFFFFF)
    key = mix(key ^ np.uint64(index))
    at = np.arange(start, start + n, dtype=np.uint64)
    h = mix((at & np.uint64(0xFFFFFFFF)) ^ key ^ (at >> np.uint64(32)))
    return torch.from_numpy((h >> np.uint64(12)).astype(np.float64) / 2 ** 20)


def spacing(y):
    """Distance of E4M3's neighbouring values at y >= 0 (from the exponent's bits: a library's power may be inexact)."""
    e = (torch.frexp(y)[1] - 1).clamp(min=-6).to(torch.int64) - 3
    return ((e + 1023) << 52).view(torch.float64)


def scales(x):
    """max(amax / 448, 2^-100) of each block, of the finite values."""
    n = x.numel()
    full = torch.zeros(-(-n // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    full[:n] = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).abs()
    return (full.view(-1, BLOCK).amax(1) / 448).clamp(min=2.0 ** -100)


def check8(state, want, rounded_up=None, terms=None):
    """A State8 against its float64 moment (or root).

    The second moment is right to 6 roundings (its terms are positive), the root and the
    division by the scale to two more each: 8 half steps of float32, 2^-21, are granted to
    what is rounded.  A first moment is a sum of two terms, each right to two roundings,
    that may cancel: 4 half steps of `terms`, the sum of their magnitudes, are granted to it
    besides.  `rounded_up`: the dither; else to nearest."""
    n = want.numel()
    s = scales(want)
    got_s = state.scale.double()
    off = torch.zeros_like(want) if terms is None else 2.0 ** -22 * terms
    most = torch.zeros(s.numel() * BLOCK, dtype=torch.float64, device=want.device)
    most[:n] = off.nan_to_num(posinf=0.0)
    assert torch.all((got_s - s).abs() <= 2.0 ** -21 * s + most.view(-1, BLOCK).amax(1) / 448)
    off = off / got_s.repeat_interleave(BLOCK)[:n]
    y = want / got_s.repeat_interleave(BLOCK)[:n]
    got = state.data.flatten().double()
    ok = torch.isfinite(want)
    assert torch.all(torch.isnan(got[~ok]))
    y, got, off = y[ok], got[ok], off[ok]
    step = spacing(y.abs())
    slack = 2.0 ** -21 * y.abs() + 2.0 ** -29 + off        # (below 2^-6 float32's own subnormals count)
    if rounded_up is None:
        # half the distance to a neighbour; at a power of two the distance below is half of that above
        assert torch.all((got - y).abs() <= step / 2 + slack)
        return
    u = rounded_up.to(want.device)[ok]
    low = torch.floor((y - slack).clamp(min=0) / step + u) * step
    high = torch.floor((y + slack) / step + u) * step
    low, high = (torch.where(y > 0, x.clamp(2.0 ** -9, 448), torch.zeros_like(x)) for x in (low, high))
    # next to a power of two the two sides' steps differ: the neighbour above is granted there
    edge = (torch.log2(y.clamp(min=1e-300)) - torch.round(torch.log2(y.clamp(min=1e-300)))).abs() < 2.0 ** -20
    assert torch.all(((got >= low) & (got <= high)) | (edge & ((got - y).abs() <= step)))
