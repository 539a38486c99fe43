"""MXFP4 in 64 bits, written from the format's definition (E2M1 elements, one
E8M0 scale per 32 columns), for the tests."""
import numpy as np
import torch

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def scale_exponents(v):
    """max(floor(log2 amax) - 2, -127) of each block of 32 columns of v [..., C] (fp64)."""
    a = np.abs(v.reshape(v.shape[:-1] + (v.shape[-1] // 32, 32))).max(-1)
    m, e = np.frexp(a)  # a = m 2^e, 0.5 <= m < 1
    return np.where(a > 0, np.maximum(e - 3, -127), -127).astype(np.int64)


def round_codes(v, s):
    """E2M1 codes (0..15) of v [..., C] for block exponents s [..., C/32]; ties to the even code, beyond 6 to 6."""
    y = np.abs(v.reshape(v.shape[:-1] + (v.shape[-1] // 32, 32))) * np.exp2(-s.astype(np.float64))[..., None]
    lo = np.clip(np.searchsorted(GRID, y, side="right") - 1, 0, 7)
    hi = np.minimum(lo + 1, 7)
    mid = (GRID[lo] + GRID[hi]) / 2
    up = (y > mid) | ((y == mid) & (lo % 2 == 1))
    code = np.where((hi > lo) & up, hi, lo)
    return (code + 8 * np.signbit(v).reshape(code.shape)).reshape(v.shape).astype(np.uint8)


def values(code, s):
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    return (v.reshape(v.shape[:-1] + (v.shape[-1] // 32, 32)) * np.exp2(s.astype(np.float64))[..., None]).reshape(v.shape)


def fake(v, s=None):
    s = scale_exponents(v) if s is None else s
    return values(round_codes(v, s), s)


def unpack(data):
    """Codes [..., C] of packed bytes [..., C / 2]."""
    out = np.empty(data.shape[:-1] + (2 * data.shape[-1],), dtype=np.uint8)
    out[..., 0::2], out[..., 1::2] = data & 15, data >> 4
    return out


def untile(scales, cols, rows_of_groups):
    """Scale bytes [rows, cols / 32] of the rows of all groups in order, from the tiled layout, byte by byte."""
    stages = -(-cols // 256)
    out, tile = [], 0
    for n in rows_of_groups:
        r = np.arange(n)[:, None]
        b = np.arange(cols // 32)[None, :]
        q, i = tile + r // 128, r % 128
        out.append(scales[(q * stages + b // 8) * 1024 + b // 4 % 2 * 512 + i % 32 * 16 + i // 32 * 4 + b % 4])
        tile += 2 * -(-n // 256)
    return np.concatenate(out) if out else np.zeros((0, cols // 32), np.uint8)


def dense64(q, rows_of_groups=None):
    """The fp64 values of a package MXTensor, read through the documented layout."""
    data, sc = q.data.cpu().numpy(), q.scales.cpu().numpy()
    flat = data.reshape(-1, data.shape[-1])
    if rows_of_groups is None:
        rows_of_groups = [data.shape[-2]] * (data.shape[0] if data.ndim == 3 else 1)
    n = sum(rows_of_groups)
    s = untile(sc, 2 * data.shape[-1], rows_of_groups).astype(np.int64) - 127
    v = values(unpack(flat[:n]), s)
    return v.reshape(data.shape[:-1] + (-1,)) if n == flat.shape[0] else v


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()
