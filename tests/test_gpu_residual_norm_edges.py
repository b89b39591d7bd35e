"""residual_norm and its backward pass at flat rows far from zero, where what lies past the
last column must not reach a row's sums."""
import pytest
import torch

import muon_newton_schulz_step_amd as mn
from gpu_helpers import announce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def randn(*shape, seed=0, std=1.0, dtype=FP32):
    g = torch.Generator(DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


# (columns, a power of two, eps): the mean times 1 / sqrt(eps) is past fp32's range, a
# row's sum is not.  Each wave's share of the columns is a power of two, so that its
# mean is the value itself: one rounded in its last digit leaves deviations whose squares
# are past the range as well.
FLAT = [(4, 2.0 ** 121, 1e-5), (64, 2.0 ** 121, 1e-5), (768, 2.0 ** 112, 1e-12), (1280, 2.0 ** 112, 1e-12),
        (2050, 2.0 ** 112, 1e-12), (5120, 2.0 ** 112, 1e-12), (9216, 2.0 ** 112, 1e-12)]


@pytest.mark.parametrize("xt,bt", [(BF16, BF16), (FP32, BF16), (FP32, FP32)])
@pytest.mark.parametrize("cols,top,eps", FLAT)
def test_flat_branch(cols, top, eps, xt, bt):
    """A flat row's deviations are zeros: the branch's norm gives post_bias, h the norm of
    a finite row, and the gradients those of rows of zeros."""
    announce("residual_norm: flat branch", cols, top, xt, bt)
    rows = 6
    b = torch.full((rows, cols), top, device=DEV)
    b[1], b[2], b[4] = -top, 3.0, 0.0
    b = b.to(bt)
    x, w, pw, pb = (randn(*s, seed=i) for i, s in enumerate(((rows, cols), (cols,), (cols,), (cols,))))
    x = x.to(xt)
    zero = torch.zeros_like(b)
    for out in (BF16, FP32, E4M3):
        r, h, st = mn.residual_norm(x, b, w, w, post_weight=pw, post_bias=pb, eps=eps, out_dtype=out)
        r0, h0, st0 = mn.residual_norm(x, zero, w, w, post_weight=pw, post_bias=pb, eps=eps, out_dtype=out)
        assert torch.isfinite(r).all() and torch.equal(r, r0) and torch.equal(st[:2], st0[:2])
        assert torch.equal(st[2], b[:, 0].float())
        same = (h.data.view(torch.uint8), h0.data.view(torch.uint8)) if out == E4M3 else (h, h0)
        assert torch.equal(*same)
    dr, dh = randn(rows, cols, seed=8, dtype=xt), randn(rows, cols, seed=9, dtype=bt)
    kw = dict(post_weight=pw, post_bias=pb)
    got = mn.residual_norm_backward(dr, dh, r, b, w, st, **kw)
    ref = mn.residual_norm_backward(dr, dh, r0, zero, w, st0, **kw)
    assert all(torch.isfinite(p).all() for p in got if p is not None)
    assert all(p is q or torch.equal(p, q) for p, q in zip(got, ref))


@pytest.mark.parametrize("xt", [BF16, FP32])
@pytest.mark.parametrize("cols,top,eps", FLAT)
def test_flat_stream(cols, top, eps, xt):
    """The same for the residual stream: h is the bias, and backward as for rows of zeros."""
    announce("residual_norm: flat stream", cols, top, xt)
    rows = 6
    x = torch.full((rows, cols), top, device=DEV)
    x[1], x[2], x[4] = -top, 3.0, 0.0
    x = x.to(xt)
    w, b = randn(cols, seed=1), randn(cols, seed=2)
    zero = torch.zeros_like(x)
    branch = torch.zeros(rows, cols, dtype=xt, device=DEV)
    gate = randn(cols, seed=5)
    dr, dh = randn(rows, cols, seed=8, dtype=xt), randn(rows, cols, seed=9, dtype=xt)
    for g in (None, gate):
        r, h, st = mn.residual_norm(x, branch, w, b, gate=g, eps=eps, out_dtype=FP32)
        assert torch.equal(r, x) and torch.equal(h, b.expand(rows, -1)) and torch.equal(st[0], x[:, 0].float())
        _, _, st0 = mn.residual_norm(zero, branch, w, b, gate=g, eps=eps, out_dtype=FP32)
        got = mn.residual_norm_backward(dr, dh, r, branch, w, st, gate=g)
        ref = mn.residual_norm_backward(dr, dh, zero, branch, w, st0, gate=g)
        assert all(torch.isfinite(p).all() for p in got if p is not None)
        assert all(p is q or torch.equal(p, q) for p, q in zip(got, ref))
