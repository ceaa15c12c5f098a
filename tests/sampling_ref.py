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


# --------------------------------------------------------------------- sampling
def sample(x, uniform, temperature=None, top_k=None, top_p=None, min_p=None):
    """(tokens, log probabilities, kept, how near a decision is to its border, relative to the weights it is about) of rows x [n, vocab]
    in 64 bits."""
    n, vocab = x.shape
    tokens, logp, kept, near = np.full(n, -1), np.full(n, -np.inf), np.zeros(n, int), np.ones(n)
    for i in range(n):
        t = 1.0 if temperature is None else float(temperature[i])
        k = 0 if top_k is None else int(top_k[i])
        p = 1.0 if top_p is None else float(top_p[i])
        low = 0.0 if min_p is None else float(min_p[i])
        row = np.asarray(x[i], np.float64)
        live = row > -np.inf
        if not live.any():
            continue
        m = row.max()
        if t == 0:
            tokens[i], logp[i], kept[i] = int(np.argmax(row)), 0.0, 1
            continue
        with np.errstate(over="ignore", invalid="ignore"):
            z = np.where(live, (row - m) / t, -np.inf)
        w = np.exp(z)
        if 0 < k < vocab:
            live &= row >= np.partition(row, vocab - k)[vocab - k]
        if p < 1:
            levels, which = np.unique(row[live], return_inverse=True)
            mass = np.bincount(which, w[live])
            above = mass[::-1].cumsum()[::-1] - mass
            above[-1] = 0
            total = mass.sum()
            fits = above < p * total
            fits[-1] = True
            near[i] = min(near[i], np.abs(above[above > 0] / total - p).min(initial=1.0))
            live &= row >= levels[fits].min()
        if low > 0:
            with np.errstate(divide="ignore"):
                near[i] = min(near[i], np.abs(z[live & (z < 0)] - np.log(low)).min(initial=1.0))
            live &= w >= low
        w = np.where(live, w, 0)
        upto = w.cumsum()
        total = upto[-1]
        at = float(uniform[i]) * total
        tokens[i] = int(np.argmax(upto > at))
        inside = np.abs(upto[live] - at) / total
        near[i] = min(near[i], inside.min())
        logp[i] = z[tokens[i]] - np.log(total)
        kept[i] = live.sum()
    return tokens, logp, kept, near
