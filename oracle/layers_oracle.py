"""64-bit numpy oracle of the 8-bit linear layer and layer norm (test
infrastructure; shares no code with the GPU path)."""
from __future__ import annotations

import numpy as np

MIN_EXP = -117


def block_exponents(x, block_rows):
    """e per block of block_rows x 128: the smallest integer >= MIN_EXP with
    max |x| <= 448 * 2^e over the block's finite values."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    br, bc = -(-rows // block_rows), -(-cols // 128)
    e = np.empty((br, bc), np.int64)
    for i in range(br):
        for j in range(bc):
            top = a[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128].max()
            k = MIN_EXP
            while top > 448.0 * 2.0 ** k:  # exact: powers of two
                k += 1
            e[i, j] = k
    return e


def round_e4m3(v):
    """v to e4m3, nearest even; |v| <= 448.  Infinities and NaN give NaN."""
    v = np.asarray(v, np.float64)
    _, ex = np.frexp(np.where(np.isfinite(v), v, 1.0))  # |v| in [2^(ex-1), 2^ex)
    step = np.ldexp(1.0, np.maximum(ex - 1, -6) - 3)
    with np.errstate(invalid="ignore"):
        q = np.rint(v / step) * step  # exact but for the rint, which ties to even
    return np.where(np.isfinite(v), q, np.nan)


def expand(e, shape, block_rows):
    """Block exponents as scales 2^e, one per element."""
    s = np.ldexp(1.0, e)
    return np.repeat(np.repeat(s, block_rows, 0)[:shape[0]], 128, 1)[:, :shape[1]]


def quantize8(x, block_rows):
    """(e4m3 numbers, exponents) of a matrix.  Where e = 120 numbers stop at
    240: 256 * 2^120 is not a number of fp32 or bf16."""
    x = np.asarray(x, np.float64)
    e = block_exponents(x, block_rows)
    scale = expand(e, x.shape, block_rows)
    q = round_e4m3(x / scale)
    return np.where(scale == 2.0 ** 120, np.clip(q, -240.0, 240.0), q), e


def layer_norm(x, w, b, eps):
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    return (x - mean[:, None]) * rstd[:, None] * w + b, mean, rstd


def layer_norm_backward(dy, x, w, mean, rstd):
    """dx, dw, db with the forward pass's mean and rstd."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    xh = (x - np.asarray(mean, np.float64)[:, None]) * np.asarray(rstd, np.float64)[:, None]
    g = dy * w
    dx = np.asarray(rstd, np.float64)[:, None] * (
        g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)
