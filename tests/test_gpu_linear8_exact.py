"""Exact products of linear8 on the GPU: operands whose sums change where the 8-bit
matrix instruction cuts (13 bits below the largest product of a group).

Whole numbers up to 2, and every 32nd column 256 in a, +-256 in b, so that its products
of 2^16 cancel with those of the column 32 further on.  A cut drops the small products
beside a large one; exact ones add up, in any order, to a whole number: every partial
sum is one below 2^24 and an fp32 number.  The exact z, y and 8 bits have to come out."""
import numpy as np
import pytest
import torch

import muon_newton_schulz_step_amd as mn
from gpu_helpers import announce, to64
from oracle import layers_oracle as lo

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def whole(*shape, seed=0, top=2):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g, device=DEV).to(FP32)


def operands(m, n, k, seed=0):
    a, b = whole(m, k, seed=seed), whole(n, k, seed=seed + 1)
    for c in range(3, k - 32, 64):
        sign = 2 * torch.randint(0, 2, (n,), generator=torch.Generator(DEV).manual_seed(seed + c), device=DEV) - 1.0
        a[:, c], a[:, c + 32], b[:, c], b[:, c + 32] = 256.0, 256.0, 256.0 * sign, -256.0 * sign
    return mn.quantize8(a), mn.quantize8(b, 128), to64(a) @ to64(b).T


def rounded(x, dtype):
    return to64(torch.from_numpy(x).to(dtype).float())  # 64 bits to the type: one rounding


def check(got, kept, z, out):
    """relu2's results and the z kept are those of the exact z, rounded once."""
    kind = FP32 if out == FP32 else BF16
    assert kept.dtype == kind and np.array_equal(to64(kept), rounded(z, kind))
    y = lo.activation(z, "relu2")
    if out == E4M3:
        q, e = lo.quantize8(y, 1)
        assert np.array_equal(got.scale.cpu().numpy()[:, :e.shape[1]].astype(np.int64) - 127, e)
        assert np.array_equal(to64(got.data.float())[:, :got.cols], q)
    else:
        assert np.array_equal(to64(got), rounded(y, out))


@pytest.mark.parametrize("m,n,k", [(1, 130, 5000), (16, 260, 1300), (17, 300, 2000), (32, 140, 5120), (33, 140, 1280),
                                   (512, 300, 1280), (300, 1300, 900), (513, 200, 512), (2100, 2050, 500),
                                   (2560, 4097, 512), (513, 300, 1290), (600, 1300, 700), (2100, 2050, 600),
                                   (8192, 4096, 520)])
def test_8_bits_are_exact_by_themselves(m, n, k):
    announce("linear8 to 8 bits, exact by itself", m, n, k)
    a, b, z = operands(m, n, k)
    check(*mn.linear8(a, b, activation="relu2", keep=True, out_dtype=E4M3), z, E4M3)
    zero = torch.zeros(n, device=DEV)
    for kw in (dict(bias=zero), dict(residual=zero.expand(m, -1).contiguous()), dict(activation="relu")):
        got = mn.linear8(a, b, out_dtype=E4M3, **kw)
        q, e = lo.quantize8(np.maximum(z, 0) if "activation" in kw else z, 1)
        assert np.array_equal(got.scale.cpu().numpy()[:, :e.shape[1]].astype(np.int64) - 127, e)
        assert np.array_equal(to64(got.data.float())[:, :n], q)


@pytest.mark.parametrize("m,n,k", [(1, 130, 5000), (32, 140, 5120), (512, 300, 1280), (513, 200, 512),
                                   (2560, 4097, 512)])
def test_plain_short_sums_and_few_rows(m, n, k):
    """On the limits up to which a plain product in 8 bits is exact by itself."""
    announce("linear8 to 8 bits, plain", m, n, k)
    a, b, z = operands(m, n, k)
    got = mn.linear8(a, b, out_dtype=E4M3)
    q, e = lo.quantize8(z, 1)
    assert np.array_equal(got.scale.cpu().numpy()[:, :e.shape[1]].astype(np.int64) - 127, e)
    assert np.array_equal(to64(got.data.float())[:, :n], q)


# every kernel and tile that the rules pick for exact products
EXACT = [(8, 520, 1300, BF16, None), (30, 20000, 300, BF16, (64, 128)), (70, 1003, 640, BF16, (64, 64)),
         (1027, 5120, 300, BF16, (64, 128)), (2048, 4096, 200, BF16, (128, 128)), (8192, 4096, 200, BF16, (256, 256)),
         (70, 1003, 640, FP32, (64, 64)), (513, 700, 1300, FP32, (64, 64)), (1027, 5120, 300, FP32, (64, 128)),
         (600, 1300, 1290, E4M3, (64, 128)),
         (2560, 4097, 600, E4M3, (128, 128)), (8192, 4096, 520, E4M3, (256, 256)), (33, 260, 1281, E4M3, (64, 128))]


@pytest.mark.parametrize("m,n,k,out,tile", EXACT)
def test_exact_by_choice(m, n, k, out, tile):
    announce("linear8 exact", m, n, k, out)
    a, b, z = operands(m, n, k, seed=m)
    mn.timing_read()
    mn.timing_enable(True)
    try:
        got = mn.linear8(a, b, activation="relu2", keep=True, out_dtype=out, exact=True)
        torch.cuda.synchronize()
        (r,) = mn.timing_read()
    finally:
        mn.timing_enable(False)
    if tile:
        pad = lambda v, t: -(-v // t) * t  # noqa: E731
        assert r["exec_flops"] == 2.0 * pad(m, tile[0]) * pad(n, tile[1]) * pad(k, 128)
    check(*got, z, out)


def test_rows_do_not_depend_on_the_batch():
    """With exact products a row is the same, whatever rows stand beside it."""
    announce("linear8 exact: batches")
    a, b, _ = operands(1100, 300, 1300, seed=5)
    x, bias = a.dequantize(FP32), torch.full((300,), 0.37, device=DEV)
    ref = mn.linear8(a, b, bias, activation="gelu", out_dtype=E4M3)
    for m in (1, 20, 512, 513):
        part = mn.linear8(mn.quantize8(x[:m].contiguous()), b, bias, activation="gelu", out_dtype=E4M3)
        assert torch.equal(part.data.view(torch.uint8), ref.data.view(torch.uint8)[:m])
        assert torch.equal(part.scale, ref.scale[:m])


# every tile that the rules pick for the 8-bit instruction's products in 8 bits
FAST = [(600, 1300, 1290, (64, 128)), (2100, 2050, 140, (128, 128)), (2560, 4097, 600, (256, 256)),
        (33, 260, 130, (64, 128))]


@pytest.mark.parametrize("m,n,k,tile", FAST)
def test_fast_by_choice(m, n, k, tile):
    """Those of a bf16 result: z of real numbers is the same, and small whole numbers, of
    which the instruction cuts nothing, give the exact 8 bits."""
    announce("linear8 to 8 bits, fast", m, n, k)
    g = torch.Generator(DEV).manual_seed(m)
    a = mn.quantize8(torch.randn(m, k, generator=g, device=DEV))
    b = mn.quantize8(torch.randn(n, k, generator=g, device=DEV), 128)
    kept = [mn.linear8(a, b, activation="silu", keep=True, out_dtype=out, exact=False)[1] for out in (BF16, E4M3)]
    assert torch.equal(*kept)
    assert torch.equal(kept[0], mn.linear8(a, b, activation="silu", keep=True)[1])
    av, bv = whole(m, k, seed=1), whole(n, k, seed=2)
    a, b, bias = mn.quantize8(av), mn.quantize8(bv, 128), whole(n, seed=3, top=9)
    res = whole(m, n, seed=4, top=50).to(BF16)
    mn.timing_read()
    mn.timing_enable(True)
    try:
        got = mn.linear8(a, b, bias, activation="relu2", residual=res, out_dtype=E4M3, exact=False)
        torch.cuda.synchronize()
        (r,) = mn.timing_read()
    finally:
        mn.timing_enable(False)
    pad = lambda v, t: -(-v // t) * t  # noqa: E731
    assert r["exec_flops"] == 2.0 * pad(m, tile[0]) * pad(n, tile[1]) * pad(k, 128)
    y = lo.activation(to64(av) @ to64(bv).T + to64(bias), "relu2") + to64(res)
    q, e = lo.quantize8(y, 1)
    assert np.array_equal(got.scale.cpu().numpy()[:, :e.shape[1]].astype(np.int64) - 127, e)
    assert np.array_equal(to64(got.data.float())[:, :n], q)
    with pytest.raises(ValueError):
        mn.linear8(a, b, out_dtype=FP32, exact=False)


@pytest.mark.parametrize("m", [7, 90, 600])
def test_operands_that_are_not_finite(m):
    """A NaN in a row of a, or of b, is in that row, or column, of every result and in no
    other place."""
    announce("linear8: NaN in an operand", m)
    n, k = 300, 1300
    av, bv = whole(m, k, seed=1), whole(n, k, seed=2)
    ref_a, ref_b = mn.quantize8(av), mn.quantize8(bv)
    av[3, 700], bv[200, 64] = float("nan"), float("inf")
    a, b = mn.quantize8(av), mn.quantize8(bv)
    keep = torch.ones(m, n, dtype=torch.bool, device=DEV)
    keep[3], keep[:, 200] = False, False
    for out in (BF16, FP32, E4M3):
        for exact in (None, True, False):
            if out == FP32 and exact is False:
                continue
            y, z = mn.linear8(a, b, activation="silu", keep=True, out_dtype=out, exact=exact)
            ref, zref = mn.linear8(ref_a, ref_b, activation="silu", keep=True, out_dtype=out, exact=exact)
            assert torch.isnan(z[~keep]).all() and torch.equal(z[keep], zref[keep])
            if out != E4M3:
                assert torch.isnan(y[~keep]).all() and torch.equal(y[keep], ref[keep])
                continue
            assert torch.isnan(y.dequantize()[~keep]).all()
            rows = keep.any(1)
            blocks = [0, 2]                                   # of the column that is not finite: the second
            assert torch.equal(y.scale[rows][:, blocks], ref.scale[rows][:, blocks])
            for c in (slice(0, 128), slice(256, 300)):
                assert torch.equal(y.data.view(torch.uint8)[rows][:, c], ref.data.view(torch.uint8)[rows][:, c])
