"""A block's fused operators and clipping where they could go wrong: special values
into 8 bits, offsets past 32 bits, vectors at any element, two graphs and two
threads at once, another stream, an infinity through every activation."""
import concurrent.futures

import numpy as np
import pytest
import torch

import muon_newton_schulz_step_amd as mn
from gpu_helpers import announce, to64
from oracle import layers_oracle as lo

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
INF, NAN = float("inf"), float("nan")


def randn(*shape, seed=0, std=1.0, mean=0.0, dtype=FP32):
    g = torch.Generator(DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * std + mean).to(dtype)


def whole(*shape, seed=0, top=2, dtype=FP32):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g, device=DEV).to(dtype)


def check8(t, ref):
    q, e = lo.quantize8(ref, 1)
    nb = e.shape[1]
    assert np.array_equal(t.scale.cpu().numpy()[:, :nb].astype(np.int64) - 127, e)
    assert np.array_equal(to64(t.data.float())[:, :t.cols], q, equal_nan=True)
    assert torch.count_nonzero(t.data.view(torch.uint8)[:, t.cols:]) == 0
    assert (t.scale[:, nb:] == 10).all()


def special(rows=129, cols=520):
    """Zeros, infinities, NaN, subnormal and the largest numbers, ties of e4m3, in blocks
    with and without ordinary values."""
    x = randn(rows, cols, seed=3)
    x[0] = 0.0
    x[1, :128] = torch.linspace(-448, 448, 128, device=DEV)
    x[2, 5], x[2, 300], x[2, 301], x[2, 519] = INF, NAN, -INF, NAN
    x[3] = NAN
    x[4] *= 1e-36
    x[5] *= 1e-42
    x[6, 17], x[6, 200], x[6, 201], x[6, 400] = 3.0e38, 1.75 * 2.0 ** 127, 2.9e38, -3.4e38
    x[7, :16] = torch.tensor([448.0, 449, 464, 17, 19, 0.5, 0.53125, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10,
                              2.0 ** -11, -17, -19, 1.0625, 1.1875, -0.0], device=DEV)
    x[8], x[8, 0] = 1e-6, 3e38
    x[9] = INF
    x[10, ::2], x[10, 1::2] = NAN, 1.0
    x[11, 100:140] = -INF
    x[12, 0::7] = NAN
    return x


@pytest.mark.parametrize("dtype", [FP32, BF16])
def test_special_values_into_8_bits(dtype):
    announce("linear8_backward: special values to 8 bits", dtype)
    dy = special().to(dtype)
    _, dz8, _ = mn.linear8_backward(dy, bias=False)
    check8(dz8, to64(dy))


@pytest.mark.parametrize("rows", [13, 129, 700])
def test_special_values_through_the_product(rows):
    """A product of zeros plus the values as the residual: few rows, and tiles."""
    announce("linear8: special values to 8 bits", rows)
    res = special(max(rows, 129))[:rows].contiguous()
    a = mn.quantize8(torch.zeros(rows, 640, device=DEV))
    b = mn.quantize8(torch.zeros(520, 640, device=DEV), 128)
    out = mn.Tensor8.empty(rows, 520, 1, DEV)
    got = mn.linear8(a, b, residual=res, out=out)
    assert got is out
    check8(out, to64(res))
    check8(mn.linear8(a, b, residual=res, out_dtype=E4M3), to64(res))


def test_special_values_of_a_norm():
    """8-bit results of rows that are not finite: NaN where the value is, and padding
    and the other rows as ever."""
    announce("residual_norm: special rows to 8 bits")
    x = randn(20, 700, seed=1)
    w, b = randn(700, seed=2, mean=1.0), randn(700, seed=3)
    ref = mn.residual_norm(x, None, w, b, out_dtype=E4M3)[1]
    bad = x.clone()
    bad[3, 5], bad[7, 699], bad[11] = INF, NAN, NAN
    h = mn.residual_norm(bad, None, w, b, out_dtype=E4M3)[1]
    good = [i for i in range(20) if i not in (3, 7, 11)]
    assert torch.equal(h.data.view(torch.uint8)[good], ref.data.view(torch.uint8)[good])
    assert torch.equal(h.scale[good], ref.scale[good])
    assert torch.count_nonzero(h.data.view(torch.uint8)[:, 700:]) == 0
    assert torch.isnan(h.dequantize()[[3, 7, 11]]).all()


@pytest.mark.parametrize("act", lo.ACTIVATIONS)
def test_infinity_through_an_activation(act):
    announce("linear8: infinite bias", act)
    for m in (3, 200):
        a, b = mn.quantize8(whole(m, 256, seed=1)), mn.quantize8(whole(140, 256, seed=2), 128)
        bias = whole(140, seed=3)
        bias[9] = INF
        for out in (BF16, FP32):
            y = mn.linear8(a, b, bias, activation=act, out_dtype=out)
            assert (y[:, 9] == INF).all() and torch.isfinite(y).sum() == y.numel() - m


def test_offsets_past_32_bits():
    announce("offsets past 2^32 bytes")
    ld, cols, rows = 1 << 30, 200, 4                  # bf16 rows 2 GiB apart
    big = torch.empty((rows - 1) * ld + cols, dtype=BF16, device=DEV)
    far = torch.as_strided(big, (rows, cols), (ld, 1))
    x = whole(rows, cols, seed=1, top=50, dtype=BF16)
    far.copy_(x)
    a, b = mn.quantize8(whole(rows, 256, seed=2)), mn.quantize8(whole(cols, 256, seed=3), 128)
    ref = mn.linear8(a, b, residual=x)
    assert torch.equal(mn.linear8(a, b, residual=far), ref)
    z = whole(rows, cols, seed=4, dtype=BF16)
    for got, want in zip(mn.linear8_backward(far, z, activation="relu2"), mn.linear8_backward(x, z, activation="relu2")):
        if isinstance(got, mn.Tensor8):
            got, want = got.data.view(torch.uint8), want.data.view(torch.uint8)
        assert torch.equal(got, want)
    w = randn(cols, seed=5)
    for branch in (far, z):
        got = mn.residual_norm(far, branch, w, post_weight=w, rms=True)
        want = mn.residual_norm(x, x if branch is far else z, w, post_weight=w, rms=True)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    got = mn.residual_norm_backward(far, far, far, far, w, want[2], post_weight=w, rms=True)
    ref = mn.residual_norm_backward(x, x, x, x, w, want[2], post_weight=w, rms=True)
    assert all(p is q or torch.equal(p, q) for p, q in zip(got, ref))
    m = 40                                            # and as a result, of the tiles
    a, n = mn.quantize8(whole(m, 256, seed=6)), 96
    big = big.new_empty((m - 1) * (1 << 26) + n)
    out = torch.as_strided(big, (m, n), (1 << 26, 1))  # 128 MiB apart: 5 GiB
    b = mn.quantize8(whole(n, 256, seed=7), 128)
    mn.linear8(a, b, activation="relu", out=out)
    assert torch.equal(out, mn.linear8(a, b, activation="relu"))


def test_many_gradients_past_32_bits():
    announce("clip: a tensor of more than 2^32 bytes")
    g = torch.zeros((1 << 31) + 12345, dtype=BF16, device=DEV)
    g[0], g[1 << 30], g[-1] = 3.0, 4.0, 12.0
    norm = mn.clip_grads([g], 6.5)
    assert float(norm) == 13.0
    assert [float(g[i]) for i in (0, 1 << 30, -1)] == [1.5, 2.0, 6.0] and int(torch.count_nonzero(g)) == 3


def test_vectors_at_any_element():
    announce("vectors at any element")
    cols = 1030
    bufs = [randn(cols + 3, seed=s) for s in range(5)]
    at = [b[k % 3 + 1:k % 3 + 1 + cols] for k, b in enumerate(bufs)]
    own = [v.clone() for v in at]
    x, br = randn(37, cols, seed=8), randn(37, cols, seed=9, dtype=BF16)

    def run(w, b, pw, pb, g):
        r, h, st = mn.residual_norm(x, br, w, b, post_weight=pw, post_bias=pb, gate=g)
        return [r, h, st, *[t for t in mn.residual_norm_backward(x, br, r, br, w, st, post_weight=pw, post_bias=pb,
                                                                 gate=g) if t is not None]]

    assert all(torch.equal(p, q) for p, q in zip(run(*at), run(*own)))
    a, b8 = mn.quantize8(whole(50, 256, seed=1)), mn.quantize8(whole(cols, 256, seed=2), 128)
    assert torch.equal(mn.linear8(a, b8, at[0], activation="silu"), mn.linear8(a, b8, own[0], activation="silu"))


def work(seed):
    """Everything that has scratch of its own, on inputs of its own."""
    x, br = randn(900, 640, seed=seed), randn(900, 640, seed=seed + 1, dtype=BF16)
    w = randn(640, seed=seed + 2)
    r, _, st = mn.residual_norm(x, br, w, post_weight=w, gate=w)
    grads = [randn(70_000, seed=seed + 3), randn(333, seed=seed + 4, dtype=BF16)]
    outs = [torch.empty_like(g) for g in grads]

    def run():
        back = mn.residual_norm_backward(x, br, r, br, w, st, post_weight=w, gate=w, bias=False)
        dz, _, db = mn.linear8_backward(br, br, activation="silu")
        norm = mn.clip_grads(grads, 1.0, out=outs)
        return [t for t in back if t is not None] + [dz, db, norm, *outs]
    return run


def test_two_graphs_at_once():
    announce("two graphs replayed at once")
    jobs = [work(100), work(200)]
    refs = [[t.clone() for t in j()] for j in jobs]
    graphs, outs = [], []
    for j in jobs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(j())
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, g in zip(streams, graphs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        for o, r in zip(outs, refs):
            assert all(torch.equal(p, q) for p, q in zip(o, r))


def test_two_threads_and_two_streams():
    announce("two threads on one stream, and on two")
    jobs = [work(300), work(400)]
    refs = [[t.clone() for t in j()] for j in jobs]
    torch.cuda.synchronize()
    for own_stream in (False, True):
        def run(k):
            stream = torch.cuda.Stream() if own_stream else torch.cuda.current_stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got = jobs[k]()
                stream.synchronize()
            return all(torch.equal(p, q) for p, q in zip(got, refs[k]))
        with concurrent.futures.ThreadPoolExecutor(2) as ex:
            assert all(ex.map(run, (0, 1)))
