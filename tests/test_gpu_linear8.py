"""linear8 and its backward pass on the GPU against the 64-bit oracle.

Two kinds of cases.  Operands of small whole numbers: every product, sum and
square on the way is a whole number below 2^24, so z, act(z) of the ReLUs and the
residual sum are exact in fp32 (the 8-bit matrix instruction cuts 13 bits below
the largest product of a group, 4, and loses nothing of a whole number), and each
result has to be the exact one rounded once: in bf16, in fp32, and in 8 bits.

And real numbers with every activation, with bounds.  u = 2^-24.  z is off by at
most D = (2 u (k + 2) + CUT8) (sum|a b| + |bias|) (as matmul8's result; CUT8 for
those from the 8-bit instruction), act(z) by D times the largest slope nearby and
by the activation's own error E:
  sigmoid(t) = 1 / (1 + exp2(-1.4427 t)): the argument is off by 3 u |t| (constant,
  product, t itself 4 u |t| for gelu_tanh's cubic), exp2 and the reciprocal by 1 ulp
  (2 u), the sum by u: relative (8 |t| + 8) u;
  Phi: 0.75e-7 by its formula, and its evaluation: x^2 off by 4 u relative, so the
  exponential by (4 x^2 + 2) u = (2 z^2 + 2) u, six roundings of the polynomial whose
  terms are up to 3.7 times their sum, 24 u: relative (2 z^2 + 40) u of the smaller
  side, plus u.
A result in bf16 adds half a step, 2^-8 of its value; one in 8 bits 2^-4, or half
a step 2^-10 of its block's scale below 2^-6 of it."""
import numpy as np
import pytest
import torch

import muon_newton_schulz_step_amd as mn
from gpu_helpers import announce, to64
from oracle import layers_oracle as lo

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24
HALF = {BF16: 2.0 ** -8, FP32: U}
CUT8 = 7 * 2.0 ** -13  # tests/test_gpu_layers.py


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def randn(*shape, seed=0, std=1.0, dtype=FP32):
    return (torch.randn(*shape, generator=gen(seed), device=DEV) * std).to(dtype)


def whole(*shape, seed=0, top=2, dtype=FP32):
    return torch.randint(-top, top + 1, shape, generator=gen(seed), device=DEV).to(dtype)


def values(t):
    q = to64(t.data.float())[:, :t.cols]
    e = t.scale.cpu().numpy().astype(np.int64)[:, :-(-t.cols // 128)] - 127
    return q * lo.expand(e, q.shape, t.block_rows)


def check8(t, ref):
    """A Tensor8 is the one that the exact matrix `ref` has, padding included."""
    q, e = lo.quantize8(ref, 1)
    nb = e.shape[1]
    assert np.array_equal(t.scale.cpu().numpy()[:, :nb].astype(np.int64) - 127, e)
    assert np.array_equal(to64(t.data.float())[:, :t.cols], q, equal_nan=True)
    assert torch.count_nonzero(t.data.view(torch.uint8)[:, t.cols:]) == 0
    assert (t.scale[:, nb:] == 10).all()


def rounded(x, dtype):
    return to64(torch.from_numpy(x).to(dtype).float())  # 64 bits to the type: one rounding


# (m, n, k): every kernel that the rules pick: few rows of one and two kinds, the
# three tiles, ragged in each direction, a k shorter than a block, several blocks
SIZES = [(1, 1, 1), (1, 130, 384), (3, 257, 129), (16, 5120, 256), (17, 640, 130), (32, 8200, 128),
         (33, 129, 515), (70, 1003, 640), (129, 384, 1), (300, 1300, 257), (513, 8000, 130),
         (2100, 2050, 140), (4099, 4000, 64), (1027, 5120, 130), (1030, 640, 530), (2048, 4096, 64), (2100, 2050, 600)]


@pytest.mark.parametrize("m,n,k,out,bm,bn", [
    (1027, 5120, 130, FP32, 64, 128), (1030, 640, 530, E4M3, 64, 128), (300, 1300, 257, E4M3, 64, 128),
    (2048, 4096, 64, E4M3, 128, 128), (2100, 2050, 600, E4M3, 128, 128), (2560, 4097, 600, E4M3, 256, 256),
    (8192, 4096, 64, E4M3, 256, 256), (2100, 2050, 140, BF16, 128, 128), (2560, 4097, 600, BF16, 256, 256),
    (70, 1003, 640, FP32, 64, 64), (2048, 4096, 64, FP32, 128, 128), (8192, 4096, 64, FP32, 256, 256)])
def test_tiles(m, n, k, out, bm, bn):
    """The sizes of these tests reach the tiles: read from the flops that a launch executes."""
    announce("linear8 tile", m, n, k, out)
    a, b = mn.quantize8(whole(m, k, seed=m), 1), mn.quantize8(whole(n, k, seed=n + 1), 128)
    mn.timing_read()
    mn.timing_enable(True)
    try:
        mn.linear8(a, b, out_dtype=out)
        torch.cuda.synchronize()
        (r,) = mn.timing_read()
    finally:
        mn.timing_enable(False)
    pad = lambda v, t: -(-v // t) * t  # noqa: E731
    assert r["kind"] == "linear8" and r["exec_flops"] == 2.0 * pad(m, bm) * pad(n, bn) * pad(k, 128)


@pytest.mark.parametrize("out", [BF16, FP32, E4M3])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_whole_numbers(m, n, k, out):
    announce("linear8 of whole numbers", m, n, k, out)
    a, b = mn.quantize8(whole(m, k, seed=m), 1), mn.quantize8(whole(n, k, seed=n + 1), 128)
    bias, res = whole(n, seed=3, top=9), whole(m, n, seed=4, top=50, dtype=BF16 if (m + n) % 2 else FP32)
    for act, with_bias, with_res, keep in ((None, True, True, False), ("relu2", True, False, True),
                                           ("relu", False, True, True), (None, False, False, False)):
        y, z = lo.linear8(values(a), values(b), to64(bias) if with_bias else None, act,
                          to64(res) if with_res else None)
        got = mn.linear8(a, b, bias if with_bias else None, activation=act,
                         residual=res if with_res else None, keep=keep, out_dtype=out)
        if keep:
            got, kept = got
            kind = FP32 if out == FP32 else BF16
            assert kept.dtype == kind and np.array_equal(to64(kept), rounded(z, kind))
        if out == E4M3:
            check8(got, y)
        else:
            assert got.dtype == out and np.array_equal(to64(got), rounded(y, out))


@pytest.mark.parametrize("out", [FP32, E4M3])
def test_whole_numbers_large_exact_tile(out):
    """256 x 256 tiles of exact products."""
    announce("linear8 of whole numbers, 256 x 256 exact tiles", out)
    m, n, k = 8192, 4096, 64
    a, b = mn.quantize8(whole(m, k, seed=1), 1), mn.quantize8(whole(n, k, seed=2), 128)
    bias, res = whole(n, seed=3, top=9), whole(m, n, seed=4, top=50, dtype=BF16)
    y, _ = lo.linear8(values(a), values(b), to64(bias), "relu2", to64(res))
    got = mn.linear8(a, b, bias, activation="relu2", residual=res, out_dtype=out)
    if out == E4M3:
        check8(got, y)
    else:
        assert np.array_equal(to64(got), y)


def slope_and_error(z, act):
    """Largest slope nearby (z itself may be off by a little), and the error E."""
    az = np.abs(z)
    if act in (None, "relu"):
        return np.ones_like(z), np.zeros_like(z)
    if act == "relu2":
        return 2 * az + 1e-2, U * z * z
    y = lo.activation(z, act)
    if act == "gelu":
        small = np.minimum(y / np.where(z == 0, 1, z), 1 - y / np.where(z == 0, 1, z))
        return np.full_like(z, 1.13), az * (0.75e-7 + U + (2 * z * z + 40) * U * np.abs(small)) + U * np.abs(y)
    t = lo._TANH * (az + 0.044715 * az ** 3) if act == "gelu_tanh" else az
    return np.full_like(z, 1.13), np.abs(y) * (8 * t + 9) * U


def check_real(m, n, k, act, out, res_type, ba=1, bb=128, seed=0):
    a = mn.quantize8(randn(m, k, seed=seed) * torch.exp2(randn(m, 1, seed=seed + 1)), ba)
    b = mn.quantize8(randn(n, k, seed=seed + 2, std=1.5 / k ** 0.5), bb)
    bias = randn(n, seed=seed + 3, std=0.5)
    res = randn(m, n, seed=seed + 4, dtype=res_type) if res_type else None
    y, z = lo.linear8(values(a), values(b), to64(bias), act, to64(res) if res_type else None)
    got, kept = mn.linear8(a, b, bias, activation=act, residual=res, keep=True, out_dtype=out) \
        if act else (mn.linear8(a, b, bias, residual=res, out_dtype=out), None)
    mag = np.abs(values(a)) @ np.abs(values(b)).T + np.abs(to64(bias))
    cut = out == BF16 and m > 16 or out == E4M3 and m > 32 and k > (1280 if m <= 512 else 512)
    dz = (2 * U * (k + 2) + (CUT8 if cut else 0.0)) * mag
    slope, err = slope_and_error(z, act)
    bound = dz * (slope + 2 * dz) + err
    if res_type:
        bound = bound + U * (np.abs(y) + bound)
    if kept is not None:
        off = np.abs(to64(kept) - z) - dz
        assert (off <= HALF[kept.dtype] * (np.abs(z) + dz)).all()
    if out == E4M3:
        scale = lo.expand(got.scale.cpu().numpy()[:, :-(-n // 128)].astype(np.int64) - 127, y.shape, 1)
        top = np.abs(y) + bound
        blocks = np.pad(top, ((0, 0), (0, -n % 128))).reshape(m, -1, 128).max(2)
        lower = np.pad(np.maximum(np.abs(y) - bound, 0), ((0, 0), (0, -n % 128))).reshape(m, -1, 128).max(2)
        s = scale[:, ::128]
        assert (lower <= 448 * s).all()                       # no smaller scale
        assert ((blocks >= 224 * s) | (s <= 2.0 ** -117)).all()  # and no larger one
        bound = bound + np.maximum(2.0 ** -4 * top, 2.0 ** -10 * scale)
        got = values(got)
    else:
        bound = bound + HALF[out] * (np.abs(y) + bound)
        got = to64(got)
    bad = ~(np.abs(got - y) <= bound)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float((np.abs(got - y) / bound).max()))


@pytest.mark.parametrize("out", [BF16, FP32, E4M3])
@pytest.mark.parametrize("act", lo.ACTIVATIONS)
def test_activations(act, out):
    for m, n, k in ((1, 300, 200), (20, 260, 300), (65, 515, 129), (700, 900, 384)):
        announce("linear8", m, n, k, act, out)
        check_real(m, n, k, act, out, (None, BF16, FP32)[(m + n) % 3])


@pytest.mark.parametrize("out", [BF16, E4M3])
def test_large_tile(out):
    announce("linear8 256 x 256 tiles", out)
    check_real(2560, 4097, 600, "gelu", out, BF16)
    check_real(1027, 260, 1283, "silu", out, None, ba=128, bb=1)
    check_real(300, 260, 1290, "relu2", out, FP32)
    check_real(1030, 640, 1300, "gelu_tanh", out, BF16)
    check_real(1027, 5120, 200, "silu", FP32, FP32)


def test_strides_and_out():
    announce("linear8 strides")
    m, n, k = 77, 200, 256
    a, b = mn.quantize8(whole(m, k, seed=1), 1), mn.quantize8(whole(n, k, seed=2), 128)
    wide = whole(m, n + 24, seed=5, top=50, dtype=BF16)
    res = wide[:, 8:8 + n]
    for dtype in (BF16, FP32):
        whole_out = torch.full((m, n + 40), 7.0, dtype=dtype, device=DEV)
        out = whole_out[:, 16:16 + n]
        got = mn.linear8(a, b, activation="relu", residual=res, out=out)
        assert got is out
        y, _ = lo.linear8(values(a), values(b), None, "relu", to64(res))
        assert np.array_equal(to64(out), rounded(y, dtype))
        assert (whole_out[:, :16] == 7).all() and (whole_out[:, 16 + n:] == 7).all()


def test_not_finite():
    """Infinities and NaN go through every output; a row without them keeps its result."""
    announce("linear8 not finite")
    for m in (5, 70):
        a, b = mn.quantize8(whole(m, 256, seed=1), 1), mn.quantize8(whole(300, 256, seed=2), 128)
        bias, res = whole(300, seed=3), whole(m, 300, seed=4)
        ref = mn.linear8(a, b, bias, activation="relu2", residual=res, out_dtype=FP32)
        bias2, res2 = bias.clone(), res.clone()
        bias2[7], res2[2, 9], res2[3, 200], res2[4, 100] = float("nan"), float("inf"), float("nan"), float("-inf")
        for out in (BF16, FP32, E4M3):
            got, z = mn.linear8(a, b, bias2, activation="relu2", residual=res2, keep=True, out_dtype=out)
            assert torch.isnan(z[:, 7]).all() and torch.isfinite(z[:, 8:]).all()
            got = got.dequantize(FP32) if out == E4M3 else got.float()
            assert torch.isnan(got[:, 7]).all() and torch.isnan(got[3, 200])
            if out == E4M3:
                assert torch.isnan(got[2, 9]) and torch.isnan(got[4, 100])
            else:
                assert got[2, 9] == float("inf") and got[4, 100] == float("-inf")
            assert torch.isfinite(got).sum() == got.numel() - m - 3
            if out == FP32:
                same = torch.isfinite(got)
                assert torch.equal(got[same], ref[same])


def test_empty():
    announce("linear8 empty")
    a, b = mn.Tensor8.empty(0, 256, device=DEV), mn.quantize8(whole(20, 256), 128)
    assert mn.linear8(a, b, activation="gelu", out_dtype=FP32).shape == (0, 20)
    y, z = mn.linear8(a, b, activation="gelu", keep=True, out_dtype=E4M3)
    assert y.shape == (0, 20) and z.shape == (0, 20)
    dz, dz8, db = mn.linear8_backward(torch.empty(0, 20, device=DEV), torch.empty(0, 20, device=DEV),
                                      activation="gelu")
    assert dz.shape == (0, 20) and dz8.shape == (0, 20) and (db == 0).all()


# ------------------------------------------------------------ backward
def grad_error(z, act):
    """The slope's own error, from the bounds above: s (1 - s) of a sigmoid is
    s - s^2, off by 3 u and by what s is."""
    az = np.abs(z)
    if act in (None, "relu"):
        return np.zeros_like(z)
    if act == "relu2":
        return np.zeros_like(z)
    if act == "gelu":
        c = np.minimum(lo.ndtr(z), lo.ndtr(-z))
        phi = np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
        return 0.75e-7 + 2 * U + (2 * z * z + 40) * U * (c + az * phi)
    tanh = act == "gelu_tanh"
    t = lo._TANH * (az + 0.044715 * az ** 3) if tanh else az
    du = lo._TANH * (1 + 3 * 0.044715 * z * z) if tanh else 1.0
    s, r = lo.expit(np.where(z < 0, -t, t)), lo.expit(np.where(z < 0, t, -t))
    ds = s * ((8 * t * r) + 8) * U                            # d s = s (1 - s) d t, and 8 roundings
    return ds * (1 + 3 * az * du) + az * du * (6 * U * s * r + 3 * U * s) + 2 * U * s


BACK = [(1, 1), (1, 515), (3, 128), (16, 257), (17, 1003), (129, 130), (1030, 520), (2051, 96)]


@pytest.mark.parametrize("dt,zt", [(BF16, BF16), (BF16, FP32), (FP32, BF16), (FP32, FP32)])
@pytest.mark.parametrize("act", lo.ACTIVATIONS)
def test_backward(act, dt, zt):
    for rows, cols in BACK:
        announce("linear8_backward", rows, cols, act, dt, zt)
        dy = (randn(rows, cols, seed=1) * torch.exp(randn(rows, 1, seed=2))).to(dt)
        z = randn(rows, cols, seed=3, std=2.0, dtype=zt)
        if cols > 100:
            z[0, :5] = torch.tensor([0.0, -0.0, 30.0, -30.0, 5.0], device=DEV)
        ref = to64(dy) * lo.activation_grad(to64(z), act)
        off = np.abs(to64(dy)) * grad_error(to64(z), act) + U * np.abs(ref)
        dz, dz8, db = mn.linear8_backward(dy, z if act else None, activation=act)
        if act is None and dt == BF16:
            assert dz is dy
        assert dz.dtype == BF16 and dz8.shape == (rows, cols)
        assert (np.abs(to64(dz) - ref) <= off + HALF[BF16] * (np.abs(ref) + off) + 2.0 ** -133).all()
        # a column's sum of `rows` terms in any order
        assert (np.abs(to64(db) - ref.sum(0)) <= (off + rows * U * (np.abs(ref) + off)).sum(0)).all()
        if act in (None, "relu", "relu2"):                    # exact in fp32 but for relu2's product
            check8(dz8, to64((dy.float() * torch.from_numpy(lo.activation_grad(to64(z), act)).float().to(DEV))))
        else:
            scale = lo.expand(dz8.scale.cpu().numpy()[:, :-(-cols // 128)].astype(np.int64) - 127, ref.shape, 1)
            e = lo.block_exponents(ref, 1)
            near = lo.expand(e, ref.shape, 1)
            assert ((scale == near) | (np.abs(np.log2(scale / near)) == 1)).all()
            assert (scale == near).mean() > 0.99
            assert (np.abs(values(dz8) - ref) <= off + np.maximum(2.0 ** -4 * (np.abs(ref) + off), 2.0 ** -10 * scale)).all()


def test_backward_options():
    announce("linear8_backward options")
    rows, cols = 333, 264
    wide = whole(rows, cols + 16, seed=1, top=9, dtype=BF16)
    dy, z = wide[:, 8:8 + cols], whole(rows, cols + 8, seed=2, dtype=FP32)[:, :cols]
    ref = to64(dy) * lo.activation_grad(to64(z), "relu2")
    dz, dz8, db = mn.linear8_backward(dy, z, activation="relu2")
    assert np.array_equal(to64(db), ref.sum(0)) and np.array_equal(to64(dz), ref)
    check8(dz8, ref)
    old = whole(cols, seed=5)
    acc = old.clone()
    _, _, got = mn.linear8_backward(dy, z, activation="relu2", dbias=acc, accumulate=True)
    assert got is acc and np.array_equal(to64(acc), to64(old) + ref.sum(0))
    _, _, got = mn.linear8_backward(dy, z, activation="relu2", dbias=acc)
    assert np.array_equal(to64(acc), ref.sum(0))
    dz2, q2, none = mn.linear8_backward(dy, z, activation="relu2", bias=False)
    assert none is None and torch.equal(dz2, dz) and torch.equal(q2.data.view(torch.uint8), dz8.data.view(torch.uint8))
    with pytest.raises(mn.MuonError):
        mn.linear8_backward(dy, z, activation="relu2", workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


def test_backward_not_finite():
    announce("linear8_backward not finite")
    dy, z = whole(40, 300, seed=1), whole(40, 300, seed=2)
    ref, _, rdb = mn.linear8_backward(dy, z, activation="relu2")
    dy2, z2 = dy.clone(), z.clone()
    z[3, 5] = 1.0
    z2[3, 5], z2[7, 100], dy2[3, 5] = 1.0, float("nan"), float("inf")
    dz, dz8, db = mn.linear8_backward(dy2, z2, activation="relu2")
    assert dz[3, 5] == float("inf") and torch.isnan(dz[7, 100])
    assert torch.isnan(dz8.dequantize()[3, 5]) and torch.isnan(dz8.dequantize()[7, 100])
    bad = torch.zeros(40, 300, dtype=torch.bool, device=DEV)
    bad[3, 5] = bad[7, 100] = True
    assert torch.equal(dz[~bad], ref[~bad])
    cols = torch.ones(300, dtype=torch.bool, device=DEV)
    cols[5] = cols[100] = False
    assert torch.equal(db[cols], rdb[cols]) and db[5] == float("inf") and torch.isnan(db[100])


def test_gradient_by_differences():
    """The whole layer's gradient against differences of its loss, in 64 bits for
    the differences: sum(y * g) over a layer whose operands are 8-bit exactly."""
    announce("linear8 gradients by differences")
    m, n, k = 24, 40, 130
    x, w = randn(m, k, seed=1), randn(n, k, seed=2, std=0.1)
    a, (b, bt) = mn.quantize8(x), mn.quantize8(w, 128, transposed=True)
    bias, g = randn(n, seed=3), whole(m, n, seed=4).to(BF16)
    for act in lo.ACTIVATIONS:
        got = mn.linear8(a, b, bias, activation=act, keep=True, out_dtype=FP32) if act else (None, None)
        dz, dz8, db = mn.linear8_backward(g, got[1], activation=act)
        dw, dx = mn.weight_grad(dz, a), mn.matmul8(dz8, bt, out_dtype=FP32)
        loss = lambda av, bv, c: float((lo.linear8(av, bv, c, act, None)[0] * to64(g)).sum())  # noqa: E731
        av, bv, c = values(a), values(b), to64(bias)
        h = 1e-5
        for r, (i, j) in enumerate(((0, 0), (7, 100), (23, 129), (11, 64))):
            eb, ea = np.zeros_like(bv), np.zeros_like(av)
            eb[i + r, j], ea[i, j] = h, h
            ec = np.zeros(n)
            ec[i] = h
            num_w = (loss(av, bv + eb, c) - loss(av, bv - eb, c)) / (2 * h)
            num_x = (loss(av + ea, bv, c) - loss(av - ea, bv, c)) / (2 * h)
            num_b = (loss(av, bv, c + ec) - loss(av, bv, c - ec)) / (2 * h)
            # dz is rounded to bf16 (2^-8 of each term), to 8 bits (2^-4) for dx;
            # the differences are off by 1e-4 at most here
            zabs = np.abs(to64(dz))
            assert abs(float(dw[i + r, j]) - num_w) <= 2.0 ** -8 * (zabs.T @ np.abs(av))[i + r, j] + 1e-3
            assert abs(float(dx[i, j]) - num_x) <= (2.0 ** -4 + 2.0 ** -7) * (zabs @ np.abs(bv))[i, j] + 1e-3
            assert abs(float(db[i]) - num_b) <= 1e-3


def test_repeats_graph_and_stream():
    announce("linear8 captured, on another stream")
    m, n, k = 300, 640, 256
    a, b = mn.quantize8(randn(m, k, seed=1)), mn.quantize8(randn(n, k, seed=2), 128)
    bias, x = randn(n, seed=3), randn(m, k, seed=5)

    def layer():
        y, z = mn.linear8(a, b, bias, activation="gelu", keep=True, out_dtype=E4M3)
        dz, dz8, db = mn.linear8_backward(z, z, activation="gelu")
        return [y.data.view(torch.uint8), y.scale, z, dz, dz8.data.view(torch.uint8), dz8.scale, db]

    ref = layer()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = layer()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(ref, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer()
    for seed in (7, 8, 9):
        mn.quantize8(randn(m, k, seed=seed), out=a)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        eager = layer()
        assert all(torch.equal(p, q) for p, q in zip(kept, eager))
    del x
