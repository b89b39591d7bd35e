"""The 8-bit linear layer and layer norm without a GPU: sizes and refusals of
the C ABI (every rejected call returns before any HIP call is made), the
binding's checks, and pins of the 64-bit oracle."""
import ctypes

import numpy as np
import pytest
import torch

import muon_newton_schulz_step_amd as mn
from muon_newton_schulz_step_amd import _lib
from oracle import layers_oracle as lo

P = 0x100000  # aligned, never dereferenced by rejected calls
INVALID, UNSUPPORTED, WORKSPACE = (mn.MUON_ERR_INVALID_ARG, mn.MUON_ERR_UNSUPPORTED,
                                   mn.MUON_ERR_WORKSPACE)
BF16, FP32 = mn.MUON_BF16, mn.MUON_FP32


def t8(k, rows=8, cols=256, block_rows=1, data=None, scale=None):
    """A tensor8 at the k-th place of its own."""
    return _lib.MuonTensor8(P * 64 * k if data is None else data,
                            P * 64 * k + P if scale is None else scale, rows, cols, block_rows)


@pytest.mark.parametrize("rows,cols,block_rows,data,scale", [
    (1, 1, 1, 128, 4), (3, 128, 1, 384, 12), (3, 129, 128, 768, 4), (129, 513, 128, 129 * 640, 16),
    (5, 1283, 1, 5 * 1408, 5 * 12), (0, 128, 1, 0, 0), (8, 0, 1, 0, 0), (-1, 8, 1, 0, 0),
    (1 << 30, 1 << 22, 1, 1 << 52, 1 << 45), (1, (1 << 22) + 1, 1, 0, 0),
    (2 ** 31 - 256, 1, 1, (2 ** 31 - 256) * 128, (2 ** 31 - 256) * 4), (2 ** 31 - 255, 1, 1, 0, 0),
])
def test_sizes(rows, cols, block_rows, data, scale):
    lib = mn.lib()
    assert lib.muon_tensor8_bytes(rows, cols) == data
    assert lib.muon_tensor8_scale_bytes(rows, cols, block_rows) == scale
    assert lib.muon_tensor8_scale_bytes(rows, cols, 64) == 0


def quantize(x=P, dtype=BF16, rows=8, cols=256, ldx=256, out=None, other=None):
    return mn.lib().muon_quantize8(x, dtype, rows, cols, ldx, out if out is not None else t8(1),
                                   other, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=2), INVALID), (dict(x=0), INVALID), (dict(x=P + 2), INVALID),
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(ldx=255), INVALID),
    (dict(rows=2 ** 31 - 255, out=t8(1, 2 ** 31 - 255)), INVALID),
    (dict(rows=7), INVALID), (dict(cols=255), INVALID),          # not the output's shape
    (dict(out=t8(1, block_rows=64)), INVALID), (dict(out=t8(1, data=0)), INVALID),
    (dict(out=t8(1, scale=0)), INVALID), (dict(out=t8(1, data=P * 64 + 8)), INVALID),
    (dict(out=t8(1, scale=P * 64 + 2)), INVALID),
    (dict(out=t8(1, data=P)), INVALID), (dict(out=t8(1, scale=P + 16)), INVALID),  # overlaps x
    (dict(out=t8(1, scale=P * 64)), INVALID),                     # overlaps its own values
    (dict(other=t8(2, 256, 8, 1)), INVALID), (dict(other=t8(2, 8, 256, 128)), INVALID),
    (dict(other=t8(2, 256, 8, 128)), UNSUPPORTED),                # of 1-row blocks
    (dict(out=t8(1, block_rows=128), other=t8(1, 256, 8, 128)), INVALID),  # the same memory
    (dict(rows=0, out=t8(1, rows=0)), mn.MUON_OK),                # nothing to do
    (dict(rows=0, x=0, out=t8(1, rows=0, data=0, scale=0)), mn.MUON_OK),
    (dict(rows=1 << 30, cols=1 << 22, ldx=1 << 22, 
          out=t8(0, 1 << 30, 1 << 22, data=1 << 55, scale=1 << 57)), UNSUPPORTED),  # apart, too many
])
def test_quantize8_refusals(kw, expect):
    assert quantize(**kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=5), INVALID), (dict(y=0), INVALID), (dict(y=P + 4), INVALID),
    (dict(ldy=255), INVALID), (dict(t=t8(1, cols=0)), INVALID), (dict(y=P * 64), INVALID),
    (dict(t=t8(1, rows=0)), mn.MUON_OK),
])
def test_dequantize8_refusals(kw, expect):
    a = dict(t=t8(1), y=P, dtype=BF16, ldy=256) | kw
    assert mn.lib().muon_dequantize8(a["t"], a["y"], a["dtype"], a["ldy"], None) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=5), INVALID), (dict(y=0), INVALID), (dict(y=P + 4), INVALID), (dict(ldy=15), INVALID),
    (dict(b=t8(2, 16, 257)), INVALID),                           # another length
    (dict(a=t8(1, data=0)), INVALID), (dict(b=t8(2, 16, 256, 2)), INVALID),
    (dict(y=P * 64), INVALID), (dict(y=P * 128 + P), INVALID),   # overlaps a, b's scales
    (dict(a=t8(1, rows=0)), mn.MUON_OK), (dict(b=t8(2, rows=0)), mn.MUON_OK),
])
def test_matmul8_refusals(kw, expect):
    a = dict(a=t8(1), b=t8(2, 16), y=P, dtype=BF16, ldy=16) | kw
    assert mn.lib().muon_matmul8(a["a"], a["b"], a["y"], a["dtype"], a["ldy"], None) == expect


def weight_grad(dy=P, dy_dtype=BF16, lddy=48, tokens=8, n=48, x=None, dw=P * 2, dw_dtype=FP32,
                accumulate=0, ws=0, ws_bytes=0):
    return mn.lib().muon_weight_grad(dy, dy_dtype, lddy, tokens, n, x if x is not None else t8(1),
                                     dw, dw_dtype, accumulate, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dy_dtype=3), INVALID), (dict(dw_dtype=3), INVALID), (dict(accumulate=2), INVALID),
    (dict(dy_dtype=FP32), UNSUPPORTED), (dict(dw_dtype=BF16, accumulate=1), UNSUPPORTED),
    (dict(lddy=(1 << 26) + 1, tokens=1, x=t8(1, 1), dy=P << 20), UNSUPPORTED),
    (dict(dy=0), INVALID), (dict(lddy=47), INVALID), (dict(n=0), INVALID), (dict(tokens=7), INVALID),
    (dict(tokens=-1, x=t8(1, rows=-1)), INVALID), (dict(dw=0), INVALID), (dict(dw=P + 16), INVALID),
    (dict(dw=P * 64 + 128), INVALID), (dict(x=t8(1, data=P * 64 + 4)), INVALID),
    (dict(tokens=0, x=t8(1, rows=0), accumulate=1), mn.MUON_OK),
    # many tokens of a small matrix: partial sums need a workspace
    (dict(tokens=1 << 14, x=t8(1, 1 << 14), dy=P * 1024), WORKSPACE),
    (dict(tokens=1 << 14, x=t8(1, 1 << 14), dy=P * 1024, ws=P * 4096 + 16, ws_bytes=1 << 30), WORKSPACE),
    (dict(tokens=1 << 14, x=t8(1, 1 << 14), dy=P * 1024, ws=P * 1024, ws_bytes=1 << 30), INVALID),
])
def test_weight_grad_refusals(kw, expect):
    assert weight_grad(**kw) == expect


def test_workspace_sizes():
    assert mn.weight_grad_workspace_bytes(16, 48, 256) == 0
    need = mn.weight_grad_workspace_bytes(1 << 14, 48, 256)
    assert need > 0 and need % (48 * 256 * 4) == 0
    assert mn.weight_grad_workspace_bytes(0, 48, 256) == 0
    assert mn.layer_norm_backward_workspace_bytes(500, 768) % (2 * 768 * 4) == 0
    assert mn.layer_norm_backward_workspace_bytes(500, 768) > 0
    assert mn.layer_norm_backward_workspace_bytes(1, 768) == 0
    assert mn.weight_grad_workspace_bytes(2 ** 31 - 255, 48, 256) == 0
    for bad in ((0, 768), (5, 0), (5, mn.MUON_MAX_NORM_COLS + 1), (2 ** 31 - 255, 768)):
        assert mn.layer_norm_backward_workspace_bytes(*bad) == 0


def norm(x=P, dtype=BF16, ldx=256, rows=8, cols=256, w=P * 2, b=P * 3, eps=1e-5, y=P * 4,
         y_dtype=BF16, ldy=256, y8=None, mean=P * 5, rstd=P * 6):
    return mn.lib().muon_layer_norm(x, dtype, ldx, rows, cols, w, b, eps, y, y_dtype, ldy, y8,
                                    mean, rstd, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=2), INVALID), (dict(y_dtype=2), INVALID), (dict(x=0), INVALID), (dict(x=P + 8), INVALID),
    (dict(ldx=1), INVALID), (dict(ldy=255), INVALID), (dict(cols=0), INVALID), (dict(rows=-1), INVALID),
    (dict(w=0), INVALID), (dict(w=P + 2), INVALID), (dict(b=P * 3 + 1), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(y=0), INVALID), (dict(y8=t8(1)), INVALID),              # neither, both
    (dict(y=0, y8=t8(1, block_rows=128)), INVALID), (dict(y=0, y8=t8(1, 7)), INVALID),
    (dict(mean=0), INVALID), (dict(rstd=P * 6 + 2), INVALID), (dict(mean=P * 6), INVALID),
    (dict(y=P), INVALID), (dict(mean=P * 2), INVALID), (dict(y=0, y8=t8(1, scale=P)), INVALID),
    (dict(cols=16385, ldx=16385, ldy=16385), UNSUPPORTED),
    (dict(rows=0), mn.MUON_OK),
])
def test_layer_norm_refusals(kw, expect):
    assert norm(**kw) == expect


def norm_back(dy=P, dtype=BF16, lddy=256, x=P * 2, x_dtype=BF16, ldx=256, x8=None, rows=800, cols=256,
              w=P * 3, mean=P * 4, rstd=P * 5, dx=P * 6, lddx=256, dw=P * 7, db=P * 8, accumulate=0,
              ws=P * 9, ws_bytes=P):
    return mn.lib().muon_layer_norm_backward(dy, dtype, lddy, x, x_dtype, ldx, x8, rows, cols, w,
                                             mean, rstd, dx, lddx, dw, db, accumulate, ws, ws_bytes,
                                             None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=2), INVALID), (dict(x_dtype=2), INVALID), (dict(dy=0), INVALID), (dict(x=0), INVALID),
    (dict(x8=t8(1, 800)), INVALID), (dict(x=0, x8=t8(1, 7)), INVALID),
    (dict(x=0, x8=t8(1, 800, 255)), INVALID),
    (dict(dx=0), INVALID), (dict(dx=P), INVALID), (dict(dx=P * 2), INVALID), (dict(lddx=255), INVALID),
    (dict(w=0), INVALID), (dict(dw=0), INVALID), (dict(dw=P * 3), INVALID), (dict(db=P * 7), INVALID),
    (dict(mean=0), INVALID), (dict(accumulate=-1), INVALID), (dict(dw=P * 7 + 2), INVALID),
    (dict(ws=0), WORKSPACE), (dict(ws_bytes=64), WORKSPACE), (dict(ws=P * 9 + 16), WORKSPACE),
    (dict(ws=P * 7), INVALID),
    (dict(rows=8, cols=16385, lddy=16385, ldx=16385, lddx=16385), UNSUPPORTED),
    (dict(rows=0, accumulate=1), mn.MUON_OK),
])
def test_layer_norm_backward_refusals(kw, expect):
    assert norm_back(**kw) == expect


def test_tensor8_checks():
    e4, u8 = torch.float8_e4m3fn, torch.uint8
    data, scale = torch.zeros(5, 384).to(e4), torch.zeros(5, 4, dtype=u8)
    t = mn.Tensor8(data, scale, 300)
    assert t.shape == (5, 300) and t.rows == 5 and "5 x 300" in repr(t)
    assert mn.Tensor8.empty(130, 300, 128).scale.shape == (2, 4)
    with pytest.raises(AttributeError):
        t.data = data
    for bad in (lambda: mn.Tensor8(data, scale, 200), lambda: mn.Tensor8(data, scale, 385),
                lambda: mn.Tensor8(data, scale, 0), lambda: mn.Tensor8(data, scale, 300, 2),
                lambda: mn.Tensor8(data, scale, 300, 128), lambda: mn.Tensor8(data[:4], scale, 300),
                lambda: mn.Tensor8(data[:, ::2], scale, 192),
                lambda: mn.Tensor8(data, scale[:, :3], 300)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        mn.Tensor8(data.float(), scale, 300)
    with pytest.raises(TypeError):
        mn.Tensor8(data, scale.int(), 300)


def test_binding_refuses_host_tensors_and_shapes():
    x, v = torch.zeros(4, 256), torch.zeros(256)
    t = mn.Tensor8.empty(4, 256)
    for bad in (lambda: mn.quantize8(x), lambda: mn.dequantize8(t), lambda: mn.matmul8(t, t),
                lambda: mn.weight_grad(x.bfloat16(), t), lambda: mn.layer_norm(x, v),
                lambda: mn.layer_norm_backward(x, x, v, torch.zeros(4), torch.zeros(4)),
                lambda: mn.quantize8(x[0]), lambda: mn.quantize8(x[:, ::2]),
                lambda: mn.quantize8(x[:1].expand(4, 256)), lambda: mn.quantize8(x.t()),
                lambda: mn.quantize8(x, transposed=True), lambda: mn.quantize8(x, 128, out=t),
                lambda: mn.matmul8(t, mn.Tensor8.empty(4, 128)),
                lambda: mn.matmul8(t, t, out=torch.zeros(4, 5)),
                lambda: mn.weight_grad(x[:3].bfloat16(), t), lambda: mn.weight_grad(x, t, accumulate=True),
                lambda: mn.layer_norm(x, v[:200]), lambda: mn.layer_norm(x, v.double()),
                lambda: mn.layer_norm_backward(x, x[:3], v, v[:4], v[:4]),
                lambda: mn.layer_norm_backward(x, x, v, v[:4], v[:4], accumulate=True),
                lambda: mn.layer_norm_backward(x, x, v, v[:4], v[:4], bias=False, dbias=v)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        mn.quantize8(x.half())
    with pytest.raises(TypeError):
        mn.dequantize8(t, torch.float16)


@pytest.mark.parametrize("rows,cols", [(2 ** 28 - 15, 512), (2 ** 27, 513)])
def test_more_threads_than_a_launch_has_are_refused(rows, cols):
    # (pieces of 512 columns with 16 threads each)
    far = t8(0, rows, cols, data=1 << 55, scale=1 << 57)
    assert quantize(rows=rows, cols=cols, ldx=cols, out=far) == UNSUPPORTED
    assert mn.lib().muon_dequantize8(far, P, BF16, cols, None) == UNSUPPORTED


@pytest.mark.parametrize("rows", [2 ** 31 - 255, 2 ** 32 + 5])
def test_binding_refuses_rows_past_32_bits(rows):
    # the sizes of the C ABI are ints: 2^32 + 5 rows must not pass for 5
    x = torch.empty(rows, 1, dtype=torch.bfloat16, device="meta")
    for bad in (lambda: mn.quantize8(x), lambda: mn.quantize8(x.t().contiguous()),
                lambda: mn.layer_norm(x, torch.ones(1)),
                lambda: mn.Tensor8.empty(rows, 1, device="meta"),
                lambda: mn.Tensor8(torch.empty(rows, 128, dtype=torch.float8_e4m3fn, device="meta"),
                                   torch.empty(rows, 4, dtype=torch.uint8, device="meta"), 1)):
        with pytest.raises(ValueError, match="rows"):
            bad()


def test_oracle_rounding_pins():
    # e4m3: 3 fraction bits, normal from 2^-6, step 2^-9 below, largest 448
    table = np.array([s * f * 2.0 ** e for s in (1, -1) for e in range(-6, 9)
                      for f in 1 + np.arange(8) / 8] + [s * k * 2.0 ** -9 for s in (1, -1)
                                                        for k in range(8)])
    table = table[np.abs(table) <= 448]
    assert np.array_equal(lo.round_e4m3(table), table)
    v = np.random.default_rng(0).uniform(-448, 448, 4000) * 2.0 ** np.random.default_rng(1).integers(-12, 1, 4000)
    near = np.abs(v[:, None] - table[None]).min(1)
    assert np.array_equal(np.abs(lo.round_e4m3(v) - v), near)
    assert lo.round_e4m3(np.array([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10]))\
        .tolist() == [16.0, 20.0, 0.0, 2.0 ** -8]  # ties to even
    assert np.isnan(lo.round_e4m3(np.array([np.inf, -np.inf, np.nan]))).all()
    # torch's own e4m3 conversion agrees
    assert np.array_equal(torch.tensor(v).float().to(torch.float8_e4m3fn).double().numpy(),
                          lo.round_e4m3(torch.tensor(v).float().double().numpy()))


def test_oracle_scale_pins():
    for top, e in ((448.0, 0), (448.0001, 1), (224.0, -1), (1.0, -8), (0.0, -117), (1e-45, -117),
                   (3.3895313892515355e38, 120), (0.875, -9), (0.8750001, -8)):
        assert lo.block_exponents(np.array([[top, 0.0]]), 1)[0, 0] == e, top
    x = np.array([[np.inf, 3.0, np.nan, -448.0]])
    assert lo.block_exponents(x, 1)[0, 0] == 0


def test_oracle_gradients_against_differences():
    rng = np.random.default_rng(3)
    x, dy = rng.normal(size=(5, 37)) * 2 + 1, rng.normal(size=(5, 37))
    w, b = rng.normal(size=37), rng.normal(size=37)
    _, mean, rstd = lo.layer_norm(x, w, b, 1e-5)
    grads = lo.layer_norm_backward(dy, x, w, mean, rstd)
    loss = lambda x, w, b: (dy * lo.layer_norm(x, w, b, 1e-5)[0]).sum()  # noqa: E731
    h = 1e-5
    for which, g in enumerate(grads):
        v = rng.normal(size=g.shape)
        hi, lw = [x, w, b], [x, w, b]
        hi[which], lw[which] = hi[which] + h * v, lw[which] - h * v
        diff = (loss(*hi) - loss(*lw)) / (2 * h)
        # central differences: an error of order h^2 = 1e-10 and 1e-16 / h of rounding
        assert abs(diff - (g * v).sum()) <= 1e-8 * (1 + np.abs(g * v).sum())
