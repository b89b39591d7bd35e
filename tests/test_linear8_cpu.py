"""linear8 and its backward pass without a GPU: refusals of the C ABI (every
rejected call returns before any HIP call is made), the binding's checks, and the
oracle's activations against differences."""
import ctypes

import numpy as np
import pytest
import torch

import muon_newton_schulz_step_amd as mn
from muon_newton_schulz_step_amd import _lib
from oracle import layers_oracle as lo

P = 0x100000  # aligned, never dereferenced by rejected calls
INVALID, UNSUPPORTED, WORKSPACE, OK = (mn.MUON_ERR_INVALID_ARG, mn.MUON_ERR_UNSUPPORTED,
                                       mn.MUON_ERR_WORKSPACE, mn.MUON_OK)
BF16, FP32 = mn.MUON_BF16, mn.MUON_FP32


def t8(k, rows=8, cols=256, block_rows=1, data=None, scale=None):
    return _lib.MuonTensor8(P * 64 * k if data is None else data,
                            P * 64 * k + P if scale is None else scale, rows, cols, block_rows)


def forward(a=None, b=None, bias=P, act=2, res=P * 2, rdt=BF16, ldr=16, z=P * 3, ldz=16, y=P * 4,
            dtype=BF16, ldy=16, y8=None):
    return mn.lib().muon_linear8(a or t8(1), b or t8(2, 16, 256, 128), bias, act, res, rdt, ldr, z,
                                 ldz, y, dtype, ldy, y8, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(act=-1), INVALID), (dict(act=6), INVALID), (dict(dtype=2), INVALID), (dict(rdt=2), INVALID),
    (dict(bias=P + 2), INVALID), (dict(b=t8(2, 16, 257)), INVALID), (dict(a=t8(1, data=0)), INVALID),
    (dict(y=0), INVALID), (dict(y=P * 4 + 8), INVALID), (dict(ldy=15), INVALID),
    (dict(res=P * 2 + 2), INVALID), (dict(ldr=15), INVALID), (dict(z=P * 3 + 4), INVALID),
    (dict(ldz=15), INVALID),
    (dict(y8=t8(3, 8, 16)), INVALID),                              # both results
    (dict(y=0, y8=t8(3, 8, 17)), INVALID), (dict(y=0, y8=t8(3, 7, 16)), INVALID),
    (dict(y=0, y8=t8(3, 8, 16, 128)), INVALID), (dict(y=0, y8=t8(3, 8, 16, data=0)), INVALID),
    (dict(y=P * 2), INVALID), (dict(y=P * 3), INVALID), (dict(z=P * 2), INVALID),  # overlaps
    (dict(y=P), INVALID), (dict(y=P * 64), INVALID), (dict(z=P * 64 + P), INVALID),
    (dict(y=0, y8=t8(2, 8, 16)), INVALID), (dict(y=0, z=P * 64 * 3, y8=t8(3, 8, 16)), INVALID),
    (dict(a=t8(1, 0)), OK), (dict(b=t8(2, 0)), OK), (dict(a=t8(1, 0), y=0, z=0, res=0, bias=0), OK),
    (dict(a=t8(0, 2 ** 31 - 256, 1, data=1 << 50, scale=1 << 52),
          b=t8(0, 2 ** 31 - 256, 1, data=1 << 54, scale=1 << 56), bias=0, res=0, z=0, y=1 << 20,
          ldy=2 ** 31 - 256), INVALID),                            # its y meets everything
])
def test_forward_refusals(kw, expect):
    assert forward(**kw) == expect


def backward(dy=P, dt=BF16, lddy=256, z=P * 2, zt=BF16, ldz=256, act=2, rows=8, cols=256, dz=P * 3,
             lddz=256, dz8=None, dbias=P * 4, accumulate=0, ws=P * 5, ws_bytes=1 << 20):
    return mn.lib().muon_linear8_backward(dy, dt, lddy, z, zt, ldz, act, rows, cols, dz, lddz, dz8,
                                          dbias, accumulate, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dt=2), INVALID), (dict(zt=2), INVALID), (dict(act=6), INVALID), (dict(accumulate=2), INVALID),
    (dict(dy=0), INVALID), (dict(dy=P + 2), INVALID), (dict(lddy=255), INVALID),
    (dict(z=0), INVALID), (dict(z=P * 2 + 2), INVALID), (dict(ldz=255), INVALID),
    (dict(dz=P * 3 + 2), INVALID), (dict(lddz=255), INVALID), (dict(dbias=P * 4 + 2), INVALID),
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID),
    (dict(cols=(1 << 22) + 1, lddy=1 << 23, ldz=1 << 23, lddz=1 << 23), INVALID),
    (dict(dz=0, dbias=0), INVALID),                                # nothing to compute
    (dict(dz8=t8(1, 8, 255)), INVALID), (dict(dz8=t8(1, 7, 256)), INVALID),
    (dict(dz8=t8(1, block_rows=128)), INVALID),
    (dict(dz=P), INVALID), (dict(dz=P * 2), INVALID), (dict(dbias=P * 3), INVALID),
    (dict(dz8=t8(1, data=P)), INVALID), (dict(dz8=t8(1, scale=P * 3)), INVALID),
    (dict(rows=100, ws=0), WORKSPACE), (dict(rows=100, ws=P * 5 + 16), WORKSPACE),
    (dict(rows=100, ws_bytes=7 * 1024 - 1), WORKSPACE), (dict(rows=100, ws=P * 4), INVALID),
    (dict(rows=100, ws=P), INVALID),
    (dict(rows=0, dbias=0), OK), (dict(rows=0, accumulate=1), OK), (dict(rows=0, dy=0, z=0, dz=0, dbias=0), OK),
])
def test_backward_refusals(kw, expect):
    assert backward(**kw) == expect


def test_workspace_sizes():
    f = mn.linear8_backward_workspace_bytes
    assert f(16, 5120) == 0 and f(17, 512) == 2 * 512 * 4      # two rows to a wave of eight
    assert f(1 << 20, 512) == 512 * 512 * 4 and f(1 << 20, 1 << 22) == 0
    assert f(0, 8) == f(-1, 8) == f(8, 0) == f(8, (1 << 22) + 1) == f(1 << 40, 8) == 0


def test_binding_refusals():
    a, b = mn.Tensor8.empty(8, 256, device="cpu"), mn.Tensor8.empty(16, 256, 128, device="cpu")
    for kw in (dict(activation="tanh"), dict(keep=True), dict(residual=torch.zeros(8, 15)),
               dict(bias=torch.zeros(15)), dict(bias=torch.zeros(16, dtype=torch.bfloat16)), dict()):
        with pytest.raises(ValueError):        # (the last: not on a GPU)
            mn.linear8(a, b, **kw)
    dy = torch.zeros(8, 16)
    for kw in (dict(activation="relu"), dict(activation="relu", z=torch.zeros(8, 15)),
               dict(bias=False, dbias=torch.zeros(16)), dict(accumulate=True),
               dict(dbias=torch.zeros(15)), dict(activation="x"), dict()):
        with pytest.raises(ValueError):
            mn.linear8_backward(dy, **kw)


@pytest.mark.parametrize("act", lo.ACTIVATIONS)
def test_oracle_slopes(act):
    z = np.linspace(-7.0, 7.0, 1401) + 0.0005                  # not at relu's corner
    h = 1e-6
    slope = (lo.activation(z + h, act) - lo.activation(z - h, act)) / (2 * h)
    assert np.max(np.abs(slope - lo.activation_grad(z, act))) < 1e-7
    assert lo.activation(np.zeros(1), act) == 0.0
    t = torch.from_numpy(z)
    pin = {None: t, "relu": torch.relu(t), "relu2": torch.relu(t) ** 2, "silu": torch.nn.functional.silu(t),
           "gelu": torch.nn.functional.gelu(t), "gelu_tanh": torch.nn.functional.gelu(t, approximate="tanh")}
    assert np.max(np.abs(lo.activation(z, act) - pin[act].numpy())) < 1e-12
