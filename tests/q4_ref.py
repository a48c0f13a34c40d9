"""4-bit matrices without the library: their quantization in numpy's float32, layout and values."""
import numpy as np
import torch


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)


def groups(x, group):
    """(whole numbers [n, k], bfloat16 scales) of float32 x: divisions in float32, rounded to nearest even."""
    n, k = x.shape
    g = -(-k // group)
    full = np.zeros((n, g * group), np.float32)
    full[:, :k] = x.float().cpu().numpy()
    full = full.reshape(n, g, group)
    with np.errstate(all="ignore"):
        bad = ~np.isfinite(full).all(-1)
        amax = np.abs(np.where(bad[..., None], 0, full)).max(-1)
        s = bf16(amax / np.float32(7))
        by = s.float().numpy()
        q = np.rint(full / np.where(by > 0, by, 1)[..., None])
        q = np.where((by > 0)[..., None] & ~bad[..., None], np.clip(q, -8, 7), 0)
    s[torch.from_numpy(bad)] = float("nan")
    return torch.from_numpy(q.reshape(n, -1)[:, :k].astype(np.int8)), s


def column_of_nibble(k):
    """The column of each held nibble of a row, in the order of the bits, from the layout's definition."""
    out = []
    for chunk in range(-(-k // 128)):
        for t in range(4):
            for j in range(4):
                out += [128 * chunk + 32 * j + 8 * t + c for c in (0, 2, 4, 6, 1, 3, 5, 7)]
    return out


def pack(q):
    n, k = q.shape
    cols = column_of_nibble(k)
    full = np.zeros((n, len(cols)), np.uint8)
    full[:, :k] = q.cpu().numpy().astype(np.int16) + 8
    full[:, k:] = 8
    nib = full[:, cols]
    return torch.from_numpy(nib[:, 0::2] | (nib[:, 1::2] << 4))


def unpack(data, k):
    data = data.cpu().numpy()
    nib = np.stack([data & 15, data >> 4], -1).reshape(data.shape[0], -1)
    out = np.zeros_like(nib)
    out[:, column_of_nibble(k)] = nib
    return torch.from_numpy(out.astype(np.int16) - 8)
