"""Edges of the 8-bit linear layer and layer norm on the GPU, against the 64-bit
oracle.  Bounds as in test_gpu_layers.py."""
import numpy as np
import pytest
import torch

import muon_newton_schulz_step_amd as mn
from gpu_helpers import announce, to64
from oracle import layers_oracle as lo
from test_gpu_layers import BF16, CUT8, DEV, E4M3, EPS, FP32, HALF, U, check8, parts, randn, within

pytestmark = pytest.mark.gpu

TOP = 2.0 ** 120


def largest(rows, cols, dtype):
    """Rows whose first block has values that round to 256 * 2^120, or nearly."""
    x = randn(rows, cols, seed=5)
    top = torch.finfo(dtype).max
    for i, v in enumerate((top, -top, 248 * TOP, -247 * TOP, 240 * TOP, 232 * TOP)):
        x[i % rows, 3 * i] = v
    return x.to(dtype)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_largest_values_stay_finite_in_8_bits(dtype, block_rows):
    announce("quantize8 of the largest values", dtype, block_rows)
    for rows, cols in ((1, 20), (7, 520), (131, 300)):
        x = largest(rows, cols, dtype)
        t = mn.quantize8(x, block_rows)
        check8(t, x, block_rows)
        for out in (BF16, FP32):
            y = mn.dequantize8(t, out)
            assert y.isfinite().all()
            assert np.array_equal(to64(y), parts(t)[2])
        if block_rows == 128:
            t, tt = mn.quantize8(x, 128, transposed=True)
            check8(t, x, 128)
            check8(tt, x.t(), 128)
    x[0, 17], x[1, 18] = float("inf"), float("nan")  # of the same blocks
    check8(mn.quantize8(x, block_rows), x, block_rows)


def test_largest_values_of_a_layer_norm_in_8_bits():
    announce("layer_norm to 8 bits, the largest values")
    bias = largest(1, 300, FP32)[0]
    t, _, _ = mn.layer_norm(randn(5, 300, seed=1), torch.zeros(300, device=DEV), bias, eps=EPS, out_dtype=E4M3)
    check8(t, bias.expand(5, 300), 1)
    assert mn.dequantize8(t).isfinite().all()


@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("m", [7, 40, 130])
def test_products_of_the_largest_values(m, out):
    # an operand of 2^128 would be an infinity, which times a zero is NaN
    announce("products of the largest values", m, out)
    a = mn.quantize8(largest(m, 300, FP32))
    w = randn(40, 300, seed=2, std=2.0 ** -20)
    w[:, :16] *= (randn(40, 16, seed=3) > 0).float()
    w[7] = 0
    b = mn.quantize8(w)
    y = mn.matmul8(a, b, out_dtype=out)
    av, bv = parts(a)[2], parts(b)[2]
    ref, mag = av @ bv.T, np.abs(av) @ np.abs(bv).T
    bound = 2 * U * 301 * mag
    if out == BF16:
        bound = bound + (CUT8 * mag if m > 16 else 0.0)
        bound = bound + HALF[BF16] * (np.abs(ref) + bound)
    within(y, ref, bound + 1e-300)
    assert torch.count_nonzero(y[:, 7]) == 0
    announce("gradients from an activation of the largest values", m)
    dy = randn(m, 40, seed=4, std=2.0 ** -20, dtype=BF16) * (randn(m, 40, seed=6) > 0)
    dw, d = mn.weight_grad(dy, a), to64(dy)
    within(dw, d.T @ av, 2 * U * (m + 2) * (np.abs(d).T @ np.abs(av)) + 1e-300)


