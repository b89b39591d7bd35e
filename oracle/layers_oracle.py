"""64-bit numpy oracle of the 8-bit linear layer and layer norm (test
infrastructure; shares no code with the GPU path)."""
from __future__ import annotations

import numpy as np
from scipy.special import expit, ndtr

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


ACTIVATIONS = (None, "relu", "relu2", "gelu", "gelu_tanh", "silu")
_TANH = 2.0 * np.sqrt(2.0 / np.pi)  # (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))


def activation(z, act):
    z = np.asarray(z, np.float64)
    if act is None:
        return z
    if act == "relu":
        return np.maximum(z, 0.0)
    if act == "relu2":
        return np.maximum(z, 0.0) ** 2
    if act == "gelu":
        return z * ndtr(z)
    return z * expit(_TANH * (z + 0.044715 * z ** 3) if act == "gelu_tanh" else z)


def activation_grad(z, act):
    """The activation's slope; relu's is 0 at 0."""
    z = np.asarray(z, np.float64)
    if act is None:
        return np.ones_like(z)
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "relu2":
        return 2.0 * np.maximum(z, 0.0)
    if act == "gelu":
        return ndtr(z) + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    u, du = (_TANH * (z + 0.044715 * z ** 3), _TANH * (1 + 3 * 0.044715 * z * z)) \
        if act == "gelu_tanh" else (z, 1.0)
    return expit(u) + z * expit(u) * expit(-u) * du


def linear8(av, bv, bias, act, residual):
    """(y, z) of the values of two 8-bit tensors."""
    z = av @ bv.T + (0.0 if bias is None else np.asarray(bias, np.float64))
    y = activation(z, act)
    return (y if residual is None else y + np.asarray(residual, np.float64)), z


def _norm(v, rms, eps):
    """(v - mean) rstd, mean, rstd of each row; a mean of 0 for RMS norm."""
    mean = np.zeros(v.shape[0]) if rms else v.mean(1)
    c = v - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(1) + eps)
    return c * rstd[:, None], mean, rstd


def _or(v, otherwise):
    return otherwise if v is None else np.asarray(v, np.float64)


def residual_norm(x, branch, w, b=None, pw=None, pb=None, gate=None, scale=None, rms=False,
                  eps=1e-5):
    """(r, h, stats of 4 x rows)."""
    x = np.asarray(x, np.float64)
    pmean = prstd = np.zeros(x.shape[0])
    p = 0.0
    if branch is not None:
        p = np.asarray(branch, np.float64)
        if pw is not None:
            p, pmean, prstd = _norm(p, rms, eps)
            p = p * pw + _or(pb, 0.0)
    r = _or(scale, 1.0) * x + _or(gate, 1.0) * p
    rh, mean, rstd = _norm(r, rms, eps)
    return r, rh * w + _or(b, 0.0), np.stack((mean, rstd, pmean, prstd))


def residual_norm_backward(dr, dh, r, branch, w, stats, x=None, pw=None, pb=None, gate=None,
                           scale=None, rms=False):
    """Gradients by name, with the forward pass's statistics."""
    dh, r = np.asarray(dh, np.float64), np.asarray(r, np.float64)
    st = np.asarray(stats, np.float64)[:, :, None]

    def back(g, vh, rstd):
        out = g - vh * (g * vh).mean(1, keepdims=True)
        return rstd * (out if rms else out - g.mean(1, keepdims=True))

    rh = (r - st[0]) * st[1]
    d = _or(dr, 0.0) + back(dh * w, rh, st[1])
    out = dict(dx=_or(scale, 1.0) * d, dweight=(dh * rh).sum(0), dbias=dh.sum(0))
    if scale is not None:
        out["dscale"] = (d * np.asarray(x, np.float64)).sum()
    if branch is None:
        return out
    bh = np.asarray(branch, np.float64)
    if pw is not None:
        bh = (bh - st[2]) * st[3]
    g = _or(gate, 1.0)
    out["dgate"] = (d * (bh * _or(pw, 1.0) + _or(pb, 0.0))).sum(0)
    if pw is None:
        out["dbranch"] = d * g + np.zeros_like(bh)
    else:
        out["dpost_weight"], out["dpost_bias"] = (g * d * bh).sum(0), (g * d).sum(0)
        out["dbranch"] = back(d * g * pw, bh, st[3])
    return out
