"""residual_norm_backward's gradient of the scale has more digits than sums in fp32."""
import numpy as np
import pytest
import torch

import muon_newton_schulz_step_amd as mn
from gpu_helpers import announce, to64
from test_scale_gradient_cpu import cancelling

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32


def randn(*shape, seed=0, dtype=FP32):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("xt,bt,top", [(FP32, FP32, 1 << 11), (FP32, BF16, 1 << 11), (BF16, BF16, 1 << 8)])
@pytest.mark.parametrize("rows,cols", [(40, 500), (4000, 200), (2000, 1280), (900, 2050), (700, 5000), (300, 9000)])
def test_cancelling_terms(rows, cols, xt, bt, top, gate):
    """Without dh, d is dr, and with odd whole numbers every product d x and pair of them
    is an fp32 number, but sums of more of them are not.  The terms cancel but for 2 x of
    one element, so that anything that a rounded sum lost on the way shows."""
    announce("residual_norm_backward: the scale's gradient", rows, cols, xt, bt, gate)
    dr, x = (torch.from_numpy(v).to(DEV).to(xt) for v in cancelling(rows, cols, top))
    dh = torch.zeros(rows, cols, dtype=bt, device=DEV)
    branch, w = randn(rows, cols, seed=1, dtype=bt), randn(cols, seed=2)
    kw = dict(gate=randn(cols, seed=3)) if gate else {}
    scale = torch.full((1,), 0.5, device=DEV)
    r, _, st = mn.residual_norm(x, branch, w, scale=scale, rms=True, **kw)
    got = mn.residual_norm_backward(dr, dh, r, branch, w, st, x=x, scale=scale, rms=True, bias=False, **kw)
    assert float(got.dscale) == 2.0 * float(x[rows // 3, cols // 2])
    assert np.array_equal(to64(got.dx), to64((0.5 * dr.float()).to(xt)))
