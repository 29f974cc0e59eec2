"""MXFP4 by its definition, in fp64.  TEST INFRASTRUCTURE ONLY."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """(codes (R, H) 0 .. 15, scales (R, H / 32) uint8) of fp32-exact values."""
    x = np.asarray(x, dtype=np.float64)
    r, h = x.shape
    b = x.reshape(r, h // 32, 32)
    finite = np.isfinite(b).all(axis=2)
    top = np.where(finite, np.abs(np.nan_to_num(b, posinf=0.0, neginf=0.0)).max(axis=2), 0.0)
    e = np.where(top > 0, np.frexp(top)[1] - 1 - 2, -127)          # floor(log2 top) - 2
    e = np.clip(e, -127, 127)
    y = np.abs(np.where(finite[..., None], b, 0.0)) / np.exp2(e.astype(np.float64))[..., None]
    y = np.minimum(y, 6.0)
    # nearest, ties to the even code: the grid's neighbours on both sides
    hi = np.clip(np.searchsorted(GRID, y), 1, 7)
    lo = hi - 1
    dl, dh = y - GRID[lo], GRID[hi] - y
    code = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    code = code + 8 * np.signbit(b)
    code = np.where(finite[..., None], code, 0)
    return code.reshape(r, h).astype(np.uint8), np.where(finite, e + 127, 255).astype(np.uint8)


def pack(code):
    return code[:, 0::2] | (code[:, 1::2] << 4)


def unpack(q):
    return np.stack((q & 15, q >> 4), axis=2).reshape(q.shape[0], -1)


def values(code, scale):
    s = np.where(scale == 255, np.nan, np.exp2(scale.astype(np.float64) - 127))
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    r, h = code.shape
    return (v.reshape(r, h // 32, 32) * s[..., None]).reshape(r, h)
