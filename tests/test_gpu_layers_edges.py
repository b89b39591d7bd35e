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


@pytest.mark.parametrize("cols", [1, 3, 130, 768, 1283, 2048, 5120, 9000, 16384])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_layer_norm_of_equal_values_gives_the_bias(cols, dtype):
    # the mean of equal values is that value, whatever its last bits: the sum's
    # rounding, d u of the value for d additions in a row (d < 64), is taken
    # off again by the sum of the deviations, which leaves d^2 u^2, below half a step
    announce("layer_norm of equal values", cols, dtype)
    v = torch.cat([torch.tensor([1000.1, -0.1, 3.3e-5, 77777.77, 1 / 3], device=DEV),
                   100 * randn(40, seed=cols)]).to(dtype)
    x = v[:, None].expand(-1, cols).contiguous()
    w, b = 1 + 0.3 * randn(cols, seed=2), 0.2 * randn(cols, seed=3)
    y, mean, rstd = mn.layer_norm(x, w, b, eps=EPS, out_dtype=FP32)
    assert torch.equal(mean, v.float())
    assert torch.equal(y, b.expand(len(v), -1))
    # no variance: the squares' mean and the correction's square are both below
    # (64 u |v|)^2; one is off by d + 3 u of that, the other by 2 (d + 3) u
    noise = 3 * 64 * U * (64 * U * np.abs(to64(v))) ** 2
    within(rstd, np.full(len(v), EPS ** -0.5), EPS ** -0.5 * (noise / EPS + 4 * U))


@pytest.mark.parametrize("cols", [768, 5120, 16384])
def test_layer_norm_of_small_variance_around_a_large_mean(cols):
    # the stored mean is the row's to half a step; y and rstd follow from it
    announce("layer_norm around a large mean", cols)
    x = 1000.1 + 1e-2 * randn(9, cols, seed=1)
    w, b = 1 + 0.3 * randn(cols, seed=2), 0.2 * randn(cols, seed=3)
    y, mean, rstd = mn.layer_norm(x, w, b, eps=EPS)
    x64, w64, b64 = to64(x), to64(w), to64(b)
    ry, rm, rr = lo.layer_norm(x64, w64, b64, EPS)
    d = 32 + 6 + 16                                   # additions in a row
    xc = np.abs(x64 - rm[:, None])
    rough = (d + 1) * U * np.abs(x64).mean(1)         # the first mean's error
    # the correction's error, and the rounding of the corrected mean
    off = (d + 2) * U * (xc.mean(1) + rough) + U * (np.abs(rm) + rough)
    within(mean, rm, off)
    # the mean square of the deviations from the first mean, var + rough^2 at
    # most, is off by d + 4 u; the square of the correction, which is taken off
    # again, by 2 rough (d + 2) u (mean |xc| + rough) <= (d + 2) u (var + 3 rough^2)
    var = (xc ** 2).mean(1)
    rel = 0.5 * 2 * (d + 5) * U * (var + 2 * rough ** 2) / (var + EPS) + 4 * U
    within(rstd, rr, rel * rr)
    dev = off[:, None] + U * xc
    by = np.abs(w64) * rr[:, None] * (dev + xc * (rel[:, None] + 4 * U)) + U * np.abs(ry)
    within(y, ry, 1.001 * by)                         # (second order)


def test_executed_flops_count_whole_tiles():
    announce("executed flops of the layers' launches")
    a, b = mn.quantize8(randn(517, 300, seed=1)), mn.quantize8(randn(771, 300, seed=2))
    mn.timing_read()
    mn.timing_enable(True)
    try:
        mn.matmul8(mn.quantize8(randn(5, 300, seed=3)), b)          # 16 x 16 to a workgroup
        mn.matmul8(a, b)                                            # 64 x 64
        mn.weight_grad(randn(517, 130, seed=4, dtype=BF16), a)      # 64 tokens, 128 x 128
        torch.cuda.synchronize()
    finally:
        mn.timing_enable(False)
    recs = [r for r in mn.timing_read() if r["kind"] in ("matmul8", "weight_grad")]
    assert [r["flops"] for r in recs] == [2.0 * 5 * 771 * 300, 2.0 * 517 * 771 * 300, 2.0 * 517 * 130 * 300]
    assert [r["exec_flops"] for r in recs] == [2.0 * 16 * 784 * 384, 2.0 * 576 * 832 * 384,
                                               2.0 * 576 * 256 * 384]


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_one_row_of_a_larger_tensor(dtype):
    # a row that begins at a multiple of 16 bytes is taken where it lies, any
    # other one refused
    announce("one row of a larger tensor", dtype)
    whole = randn(131, 389, seed=4, dtype=dtype)
    row, other = whole[8:9], whole[5:6]
    assert row.data_ptr() % 16 == 0 and other.data_ptr() % 16 != 0
    w, b = 1 + 0.3 * randn(389, seed=2), 0.2 * randn(389, seed=3)
    own = row.clone()
    for block_rows in (1, 128):
        check8(mn.quantize8(row, block_rows), row, block_rows)
    t, tt = mn.quantize8(row, 128, transposed=True)
    check8(tt, row.t(), 128)
    y, mean, rstd = mn.layer_norm(row, w, b)
    assert all(torch.equal(p, q) for p, q in zip((y, mean, rstd), mn.layer_norm(own, w, b)))
    assert all(torch.equal(p, q) for p, q in zip(mn.layer_norm_backward(row, row, w, mean, rstd),
                                                 mn.layer_norm_backward(own, own, w, mean, rstd)))
    calls = [lambda x: mn.quantize8(x), lambda x: mn.quantize8(x, 128), lambda x: mn.layer_norm(x, w, b),
             lambda x: mn.layer_norm_backward(x, own, w, mean, rstd),
             lambda x: mn.layer_norm_backward(own, x, w, mean, rstd)]
    if dtype == BF16:
        assert torch.equal(mn.weight_grad(row, t), mn.weight_grad(own, t))
        calls.append(lambda x: mn.weight_grad(x, t))
    for call in calls:
        with pytest.raises(mn.MuonError) as err:
            call(other)
        assert err.value.status == mn.MUON_ERR_INVALID_ARG
