"""References for the 8-bit activation calls, in numpy: the codes and scales of
a matrix step by step in fp32 (they are defined bit for bit), and the values,
norms and gradients in 64 bits."""
import math

import numpy as np

TOP = {"int8": np.float32(127), "e4m3": np.float32(448)}
TINY = np.float32(2.0 ** -100)
_erf = np.vectorize(math.erf, otypes=[np.float64])


def groups(cols, group):
    return -(-cols // group) if group else 1


def to_grid(v, fmt):
    """The nearest code value of v (64 bits), halves to even, saturated."""
    v = np.asarray(v, np.float64)
    if fmt == "int8":
        return np.clip(np.rint(v), -127, 127)
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    step = np.exp2(e - 3)
    return np.clip(np.rint(v / step) * step, -448, 448)


def spread(scales, cols, group):
    """Each column's scale."""
    return np.repeat(scales, group or cols, axis=-1)[..., :cols]


def pack(y, fmt, group):
    """(code values, scales) of float32 y [rows, cols]."""
    y = np.asarray(y, np.float32)
    rows, cols = y.shape
    n = groups(cols, group)
    width = group or cols
    scales = np.zeros((rows, n), np.float32)
    inv = np.zeros((rows, n), np.float32)
    for g in range(n):
        m = np.abs(y[:, g * width:(g + 1) * width]).max(1)   # NaN propagates
        with np.errstate(all="ignore"):
            s, i = m / TOP[fmt], TOP[fmt] / m
        bad = ~np.isfinite(m)
        small = ~bad & (m < TINY)
        scales[:, g] = np.where(bad, np.float32(np.nan), np.where(small, 0, s))
        inv[:, g] = np.where(bad | small, 0, i)
    iv = spread(inv, cols, group)
    with np.errstate(all="ignore"):
        codes = np.where(iv == 0, 0.0, to_grid(y * iv, fmt))
    return codes, scales


def values(codes, scales, group):
    """scale * code in fp32, as 64 bits."""
    s = spread(scales, codes.shape[-1], group)
    with np.errstate(all="ignore"):
        return (codes.astype(np.float32) * s).astype(np.float64)


def half_step(codes, scales, fmt, group):
    """Half the distance between code values around each code, in values."""
    s = spread(scales, codes.shape[-1], group).astype(np.float64)
    if fmt == "int8":
        return 0.5 * s
    e = np.floor(np.log2(np.maximum(np.abs(codes), 2.0 ** -6)))
    return s * np.exp2(e - 4)


def gelu(h):
    return 0.5 * h * (1 + _erf(h * math.sqrt(0.5)))


def gelu_slope(h):
    return 0.5 * (1 + _erf(h * math.sqrt(0.5))) + h * np.exp(-0.5 * h * h) / math.sqrt(2 * math.pi)


def rmsnorm(r, gain, eps):
    rstd = 1 / np.sqrt((r * r).mean(1) + eps)
    return r * rstd[:, None] * gain, rstd


def rmsnorm_backward(dy, r, rstd, gain, dtotal):
    """(dx, dgain) and the sums of the magnitudes that go into them."""
    n = r * rstd[:, None]
    g = dy * gain
    mean = (g * n).mean(1, keepdims=True)
    amean = np.abs(g * n).mean(1, keepdims=True)
    dx = rstd[:, None] * (g - n * mean) + dtotal
    a = rstd[:, None] * (np.abs(g) + np.abs(n) * amean) + np.abs(dtotal)
    return dx, (dy * n).sum(0), a, np.abs(dy * n).sum(0)
