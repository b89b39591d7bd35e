"""Activations and their slopes at infinities and at numbers whose squares overflow."""
import pytest
import torch

import muon_newton_schulz_step_amd as mn
from gpu_helpers import announce
from oracle import layers_oracle as lo

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
INF = float("inf")
FAR = [INF, 3.0e38, 1e25, 1.9e19, 1e10, 300.0, -300.0, -1e10, -1.9e19, -1e25, -3.0e38, -INF]


def limits(z, act):
    """(the activation, its slope) far from zero, where they are the line's or zero."""
    on = (z > 0).double()
    if act is None:
        return z, torch.ones_like(z)
    y = torch.where(z > 0, z, torch.zeros_like(z))
    return (y * y, 2 * y) if act == "relu2" else (y, on)


def far():
    """The numbers as fp32 and bf16 have them, over two blocks of columns and a ragged one."""
    return torch.tensor(FAR * 25, device=DEV)[:293].bfloat16().float()


@pytest.mark.parametrize("act", lo.ACTIVATIONS)
def test_values(act):
    announce("linear8: far from zero", act)
    z = far()
    y, _ = limits(z.double(), act)
    for m in (3, 40, 200):
        a, b = mn.quantize8(torch.zeros(m, 256, device=DEV)), mn.quantize8(torch.zeros(293, 256, device=DEV), 128)
        for out in (BF16, FP32):
            got = mn.linear8(a, b, z, activation=act, out_dtype=out)
            assert torch.equal(got, y.to(FP32).to(out).expand(m, -1)), (m, out)
        got = mn.linear8(a, b, z, activation=act, out_dtype=E4M3)
        ref = mn.quantize8(y.to(FP32).expand(m, -1).contiguous())
        assert torch.equal(got.scale, ref.scale)
        assert torch.equal(got.data.float().nan_to_num(1e9), ref.data.float().nan_to_num(1e9))


@pytest.mark.parametrize("act", lo.ACTIVATIONS)
def test_slopes(act):
    announce("linear8_backward: far from zero", act)
    z = far()
    g = torch.Generator(DEV).manual_seed(1)
    dy = torch.randint(1, 4, (20, 293), generator=g, device=DEV).to(FP32)
    ref = dy * limits(z.double(), act)[1].to(FP32)            # 2 z overflows to infinity for relu2
    for zt in (BF16, FP32):
        for dt in (BF16, FP32):
            dz, dz8, db = mn.linear8_backward(dy.to(dt), z.to(zt).expand(20, -1).contiguous(), activation=act)
            assert torch.equal(dz, ref.to(BF16))
            want = mn.quantize8(ref)
            assert torch.equal(dz8.scale, want.scale)
            assert torch.equal(dz8.data.float().nan_to_num(1e9), want.data.float().nan_to_num(1e9))
            if act != "relu2":
                assert torch.equal(db, ref.sum(0))
    nan = torch.full((2, 293), float("nan"), device=DEV)
    if act is not None:
        assert torch.isnan(mn.linear8_backward(dy[:2], nan, activation=act)[0]).all()
