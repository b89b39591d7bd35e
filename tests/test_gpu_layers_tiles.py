"""Every tile of the 8-bit product and of the weight gradient, at ragged sizes
that its rule picks it for, against products in 64 bits.

Which tile ran is read from the timing log: a launch's executed flops are those
of whole tiles.  Where a refit of the rules' costs moves a size to another tile,
these tests fail, and the size has to be replaced by one that still takes it.

Bounds as in test_gpu_layers.py; the 64-bit products are torch's, of the values
that the 8-bit tensors stand for."""
import pytest
import torch

import muon_newton_schulz_step_amd as mn
from gpu_helpers import announce
from test_gpu_layers import BF16, CUT8, DEV, FP32, HALF, U, randn

pytestmark = pytest.mark.gpu


def up(size, tile):
    return -(-size // tile) * tile


SQUARE = [(64, 64), (128, 128), (256, 256)]
WIDE = [(256, 256), (256, 128), (128, 128)]


def check_tile(flops, rows, cols, summed, tile, tiles):
    """That a launch had tiles of that size; no other would give the same flops."""
    of = {t: 2.0 * up(rows, t[0]) * up(cols, t[1]) * summed for t in tiles}
    assert flops == of[tile], [t for t in tiles if of[t] == flops]
    assert list(of.values()).count(flops) == 1


def executed(kind, call):
    """The call's result and the flops that its launch of `kind` executed."""
    torch.cuda.synchronize()
    mn.timing_read()
    mn.timing_enable(True)
    try:
        out = call()
        torch.cuda.synchronize()
    finally:
        mn.timing_enable(False)
    flops = [r["exec_flops"] for r in mn.timing_read() if r["kind"] == kind]
    assert len(flops) == 1
    return out, flops[0]


def values(t):
    """What a Tensor8 stands for, in 64 bits."""
    scale = ((t.scale[:, :up(t.cols, 128) // 128].long() - 127 + 1023) << 52).view(torch.float64)
    scale = scale.repeat_interleave(t.block_rows, 0)[:t.rows].repeat_interleave(128, 1)
    return (t.data.float().double() * scale)[:, :t.cols].contiguous()


def within(got, ref, bound):
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


def product(m, n, k, ba, bb, out, tile, few=False, big=False):
    announce("matmul8 tile", tile, m, n, k, ba, bb, out)
    a = mn.quantize8(randn(m, k, seed=k) * torch.exp2(3 * randn(m, 1, seed=k + 1)), ba)
    b = mn.quantize8(randn(n, k, seed=k + 2, std=0.02), bb)
    y, flops = executed("matmul8", lambda: mn.matmul8(a, b, out_dtype=out))
    check_tile(flops, m, n, up(k, 128), tile, [(tile[0], 16), (tile[0], 32)] if few else SQUARE)
    assert (y.numel() * y.element_size() > 256 << 20) == big  # then it is stored past the cache
    av, bt = values(a), values(b).t().contiguous()
    ref = av @ bt
    mag = av.abs() @ bt.abs()
    bound = 2 * U * (k + 1) * mag
    if out == BF16:
        if not few:
            bound += CUT8 * mag
        bound += HALF[BF16] * (ref.abs() + bound)
        # the roundings to bf16 in the root mean square, as in product_case
        assert (y.double() - ref).norm() <= 2.0 ** -8 / 3 ** 0.5 * ref.norm()
    within(y, ref, bound + 1e-300)
    del ref, mag, bound
    # a strided output: the same numbers, and nothing beside them
    whole = torch.full((m + 1, n + 16), 7.0, device=DEV, dtype=out)
    mn.matmul8(a, b, out=whole[:m, 8:8 + n])
    assert torch.equal(whole[:m, 8:8 + n], y)
    assert (whole[:, :8] == 7).all() and (whole[:, 8 + n:] == 7).all() and (whole[m] == 7).all()


# 1 to 11 k-tiles: every count that the loop over four of them leaves, twice
@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("kt", range(1, 12))
def test_matmul8_256_tiles(kt, out):
    ba, bb = ((1, 128), (1, 1), (128, 128), (128, 1))[kt % 4]
    product(4077, 3890, 128 * kt - 37, ba, bb, out, (256, 256))


@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("kt", range(1, 9))
def test_matmul8_128_tiles(kt, out):
    product(4099, 1283, 128 * kt - 51, 1, 128, out, (128, 128))


@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("kt", range(1, 9))
def test_matmul8_64_tiles(kt, out):
    product(517, 771, 128 * kt - 5, 1, 128, out, (64, 64))


@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("m,n,tile", [(13, 517, (16, 16)), (13, 8200, (16, 32)), (29, 517, (32, 16)),
                                      (29, 8200, (32, 32))])
def test_matmul8_few_rows(m, n, tile, out):
    product(m, n, 1283, 1, 128, out, tile, few=True)


@pytest.mark.parametrize("m,n,k,out,tile", [
    (16380, 8200, 200, BF16, 256), (8190, 12090, 200, FP32, 256), (380, 353537, 130, BF16, 128),
    (8200, 8190, 300, FP32, 128), (63, 2140001, 128, BF16, 64), (60, 1200001, 128, FP32, 64)])
def test_matmul8_results_past_the_cache(m, n, k, out, tile):
    product(m, n, k, 1, 128, out, (tile, tile), big=True)


@pytest.mark.parametrize("out", [BF16, FP32])
def test_matmul8_256_tiles_keep_non_finite_rows_apart(out):
    announce("matmul8 256 x 256 tiles, NaN rows", out)
    m, n = 4077, 3890
    x, w = randn(m, 700, seed=1), randn(n, 700, seed=2)
    x[1, 7], x[m - 1, 699], w[300, 650] = float("inf"), float("nan"), float("nan")
    y, flops = executed("matmul8", lambda: mn.matmul8(mn.quantize8(x), mn.quantize8(w, 128), out_dtype=out))
    check_tile(flops, m, n, 768, (256, 256), SQUARE)
    bad = torch.zeros(m, n, dtype=torch.bool, device=DEV)
    bad[1], bad[m - 1], bad[:, 300] = True, True, True
    assert torch.equal(y.isnan(), bad)


# ------------------------------------------------------------ weight gradient
def gradient(tokens, n, k, tile, parts, out=FP32, block_rows=1, pad=0):
    announce("weight_grad tile", tile, tokens, n, k, parts, out, block_rows)
    dy = randn(tokens, n + pad, seed=tokens, std=1e-3, dtype=BF16)[:, :n]
    x = mn.quantize8(randn(tokens, k, seed=k) * torch.exp2(2 * randn(tokens, 1, seed=k + 1)), block_rows)
    scratch = mn.weight_grad_workspace_bytes(tokens, n, k)
    assert scratch == (4 * parts * n * k if parts > 1 else 0)
    dw, flops = executed("weight_grad", lambda: mn.weight_grad(dy, x, out_dtype=out))
    check_tile(flops, n, k, up(tokens, 64), tile, WIDE)
    d, v = dy.double().t().contiguous(), values(x)
    ref = d @ v
    bound = 2 * U * (tokens + 2) * (d.abs() @ v.abs())
    if out == BF16:
        bound += HALF[BF16] * (ref.abs() + bound)
    within(dw, ref, bound + 1e-300)
    return dy, x, dw


GRADIENTS = [
    # ragged rows, columns and tokens; even and odd numbers of token tiles
    (333, 3905, 3890, (256, 256), 1), (64, 3905, 3890, (256, 256), 1), (1, 3905, 3890, (256, 256), 1),
    (129, 3905, 3890, (256, 256), 1), (1000, 3905, 3890, (256, 256), 1),
    (6509, 259, 3587, (256, 256), 8), (16390, 1900, 1800, (256, 256), 4),
    (705, 3890, 1890, (256, 128), 1), (65, 3890, 1890, (256, 128), 1), (257, 3890, 1890, (256, 128), 1),
    (16399, 780, 890, (256, 128), 9), (9001, 580, 1090, (256, 128), 9), (4561, 3650, 1, (256, 128), 15),
    (705, 514, 515, (128, 128), 1), (2000, 1820, 1083, (128, 128), 1),
    (9001, 560, 1800, (128, 128), 3), (2000, 530, 560, (128, 128), 8)]


@pytest.mark.parametrize("out,block_rows,pad", [(FP32, 1, 0), (BF16, 128, 0), (FP32, 128, 13)])
@pytest.mark.parametrize("tokens,n,k,tile,parts", GRADIENTS)
def test_weight_grad_tiles(tokens, n, k, tile, parts, out, block_rows, pad):
    dy, x, dw = gradient(tokens, n, k, tile, parts, out, block_rows, pad)
    assert torch.equal(dw, mn.weight_grad(dy.contiguous(), x, out_dtype=out))
    if out == FP32:
        acc = torch.full((n, k), 3.0, device=DEV)
        assert mn.weight_grad(dy, x, out=acc, accumulate=True) is acc
        assert torch.equal(acc, 3.0 + dw)


@pytest.mark.parametrize("tokens,n,k", [(333, 3905, 3890), (6509, 259, 3587), (705, 3890, 1890),
                                        (16399, 780, 890)])
def test_weight_grad_tiles_read_nothing_behind_dy(tokens, n, k):
    # NaN behind the last row, and between the rows of a strided dy
    announce("weight_grad beside NaN", tokens, n, k)
    x = mn.quantize8(randn(tokens, k, seed=1))
    for pad in (0, 3):
        buf = torch.full((tokens * (n + pad) + 4096,), float("nan"), dtype=BF16, device=DEV)
        dy = buf[:tokens * (n + pad)].view(tokens, n + pad)[:, :n].copy_(randn(tokens, n, seed=2))
        dw = mn.weight_grad(dy, x)
        assert torch.equal(dw, mn.weight_grad(dy.contiguous(), x)) and dw.isfinite().all()


@pytest.mark.parametrize("tokens,n,k", [(333, 3905, 3890), (16399, 780, 890)])
def test_weight_grad_tiles_keep_non_finite_rows_apart(tokens, n, k):
    announce("weight_grad tiles, NaN", tokens, n, k)
    dy, x = randn(tokens, n, seed=1, dtype=BF16), randn(tokens, k, seed=2)
    x[tokens - 1, k - 1], dy[0, n - 1] = float("nan"), float("inf")
    dw = mn.weight_grad(dy, mn.quantize8(x))
    bad = torch.zeros(n, k, dtype=torch.bool, device=DEV)
    bad[:, k - 1], bad[n - 1] = True, True
    assert torch.equal(~dw.isfinite(), bad)
