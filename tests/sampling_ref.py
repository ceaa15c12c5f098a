"""Plain 64-bit forms of the sampling step's operators, from the definitions in include/dflash.h, on the CPU."""
import numpy as np


def to_type(x, kind):
    """float64 -> the nearest values of the type, as float64."""
    if kind == "fp16":
        return np.asarray(x, np.float16).astype(np.float64)
    x = np.asarray(x, np.float32)
    if kind == "fp32":
        return x.astype(np.float64)
    u = x.view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}  # a rounding, relative to the value


# ------------------------------------------------------------- norm and rotation
def angles(positions, turns, axes=None):
    """Angles [n, rotary_dim / 2] of positions [n] or [n_axes, n], from the table's whole numbers."""
    positions = np.atleast_2d(np.asarray(positions, np.int64))
    axes = np.zeros(len(turns), int) if axes is None else axes
    out = np.zeros((positions.shape[1], len(turns)))
    for j, t in enumerate(turns):
        for i, p in enumerate(positions[axes[j]]):
            part = int(p) * int(t) % (1 << 64)
            out[i, j] = 2 * np.pi * ((part - (1 << 64) if part >> 63 else part) / 2.0 ** 64)
    return out


def norm_rope(x, weight, eps, angle):
    """(z, size): the result for rows x [n, heads, d], and the size of the terms that each value is a sum of."""
    y = np.asarray(x, np.float64)
    if weight is not None:
        m = (y * y).mean(-1, keepdims=True) + eps
        y = np.divide(y, np.sqrt(m), out=np.zeros_like(y), where=m > 0) * weight
    h = 0 if angle is None else angle.shape[1]
    z, size = y.copy(), np.abs(y)
    if h:
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        a, b = y[..., :h], y[..., h:2 * h]
        z[..., :h], z[..., h:2 * h] = a * c - b * s, b * c + a * s
        size[..., :h] = size[..., h:2 * h] = np.abs(a) + np.abs(b)
    return z, size
