"""The gradients' norm and clipping on the GPU against 64 bits.

Bounds.  Squares are exact in fp64 up to 2^-53 of their value, and so is every
addition: the norm of n numbers is off by at most n 2^-53 of itself, and by half a
step of fp32, 2^-24, for its rounding.  c is one rounding to fp32 (2^-24) of a
quotient of such numbers, c g another, and bf16 adds 2^-8: a clipped value is
within 2^-22, and 2^-8 where it is bf16, of the exact one; fp32 and bf16
subnormals are off by up to a step of theirs, 2^-149 and 2^-133."""
import math

import pytest
import torch

import muon_newton_schulz_step_amd as mn
from gpu_helpers import announce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32
REL = {BF16: 2.0 ** -8 + 2.0 ** -22, FP32: 2.0 ** -22}
STEP = {BF16: 2.0 ** -133, FP32: 2.0 ** -149}


def randn(n, seed=0, std=1.0, dtype=FP32):
    g = torch.Generator(DEV).manual_seed(seed)
    return (torch.randn(n, generator=g, device=DEV) * std).to(dtype)


def norm64(ts):
    return math.sqrt(math.fsum(float(t.double().square().sum()) for t in ts))


def check_norm(norm, ref):
    assert norm.shape == () and norm.dtype == FP32
    assert abs(float(norm) - ref) <= 2.0 ** -23 * ref, (float(norm), ref)


def check_clipped(out, grads, c):
    for o, g in zip(out, grads):
        ref = g.double() * c
        assert o.shape == g.shape
        assert ((o.double() - ref).abs() <= REL[o.dtype] * ref.abs() + STEP[o.dtype]).all()


SETS = {
    "one": [1], "seven": [7], "tile": [16384], "ragged": [16385, 3, 16383, 8, 40000],
    "vectors": [13] * 300, "empty_among": [0, 5, 0, 0, 1003, 0],
    "more_than_a_launch": [777] * 129 + [100_003], "large": [20_000_003, 17, 9_999_999],
}


@pytest.mark.parametrize("types", ["bf16", "fp32", "mixed"])
@pytest.mark.parametrize("name", SETS)
def test_norm_and_clip(name, types):
    announce("clip", name, types)
    kinds = {"bf16": [BF16], "fp32": [FP32], "mixed": [BF16, FP32]}[types]
    grads = [randn(n, seed=i, std=0.01 * (1 + i % 5), dtype=kinds[i % len(kinds)])
             for i, n in enumerate(SETS[name])]
    kept = [g.clone() for g in grads]
    ref = norm64(grads)
    check_norm(mn.grad_norm(grads), ref)
    for limit in (0.3 * ref, 2.0 * ref):
        c = min(1.0, float(torch.tensor(limit, dtype=FP32)) / (ref + float(torch.tensor(1e-6, dtype=FP32))))
        for dtype in (None, BF16, FP32):
            # what lies around an output stays
            out = [torch.full((g.numel() + 16,), 5.0, dtype=dtype or g.dtype, device=DEV) for g in grads]
            views = [o[8:8 + g.numel()] for o, g in zip(out, grads)]
            check_norm(mn.clip_grads(grads, limit, out=views), ref)
            check_clipped(views, kept, c)
            assert all((o[:8] == 5).all() and (o[8 + g.numel():] == 5).all() for o, g in zip(out, grads))
        assert all(torch.equal(g, k) for g, k in zip(grads, kept))
    check_norm(mn.clip_grads(grads, 2.0 * ref), ref)
    assert all(torch.equal(g, k) for g, k in zip(grads, kept))  # not clipped: not changed
    check_norm(mn.clip_grads(grads, 0.3 * ref), ref)
    check_clipped(grads, kept, 0.3 * ref / (ref + 1e-6))


def test_views_of_a_flat_buffer():
    announce("clip", "views at every element")
    for dtype in (BF16, FP32):
        flat = randn(60_000, seed=3, dtype=dtype)
        kept = flat.clone()
        grads = [flat[i * 3001 + i:i * 3001 + i + 2990] for i in range(16)]  # 11 apart, at any element
        ref = norm64(grads)
        check_norm(mn.clip_grads(grads, 0.5 * ref), ref)
        inside = torch.zeros(60_000, dtype=torch.bool, device=DEV)
        for i in range(16):
            inside[i * 3001 + i:i * 3001 + i + 2990] = True
        assert torch.equal(flat[~inside], kept[~inside])
        check_clipped([flat[inside]], [kept[inside]], 0.5 * ref / (ref + 1e-6))


def test_extremes():
    """Squares far outside of fp32's range, subnormal numbers, zeros."""
    announce("clip", "extremes")
    for value in (3e38, 1e30, 1e-30, 1e-42, 0.0):
        g = torch.full((3, 1001), value, device=DEV)
        ref = norm64([g])
        got = mn.grad_norm([g])
        if ref > 3.4e38:
            assert math.isinf(float(got))
        else:  # a subnormal result is within a step of its own
            assert abs(float(got) - ref) <= 2.0 ** -23 * ref + 2.0 ** -149
        before = g.clone()
        mn.clip_grads([g], 1.0)
        check_clipped([g], [before], min(1.0, 1.0 / (ref + 1e-6)))


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_not_finite(bad):
    announce("clip", bad)
    a, b = randn(5000, seed=1), randn(333, seed=2, dtype=BF16)
    b[17] = bad
    norm = mn.clip_grads([a, b], 1.0)
    if bad != bad:
        assert torch.isnan(norm) and torch.isnan(a).all() and torch.isnan(b).all()
    else:
        assert torch.isinf(norm) and (a == 0).all()
        assert torch.isnan(b[17]) and (b[:17] == 0).all() and (b[18:] == 0).all()


def test_zero_limit_and_all_empty():
    announce("clip", "zero limit, empty tensors")
    a = randn(100)
    mn.clip_grads([a], 0.0)
    assert (a == 0).all()
    e = torch.empty(0, 5, device=DEV)
    assert float(mn.grad_norm([e, e])) == 0.0 and float(mn.clip_grads([e], 1.0)) == 0.0


def test_refusals():
    announce("clip", "refusals")
    a = randn(64).view(8, 8)
    for bad, err in (([a.t()], ValueError), ([a[:, :4]], ValueError), ([a.double()], TypeError),
                     ([a, a.cpu()], ValueError), ([a, a], mn.MuonError), ([a, a[2:]], mn.MuonError)):
        kept = a.clone()
        with pytest.raises(err):
            mn.clip_grads(bad, 1.0)
        assert torch.equal(a, kept)
    for kw in (dict(out=[]), dict(out=[a[:4]]), dict(out=[a.view(-1)]), dict(workspace=a.t())):
        with pytest.raises(ValueError):
            mn.clip_grads([a], 1.0, **kw)
    for limit in (-1.0, float("nan"), float("inf")):
        with pytest.raises(mn.MuonError):
            mn.clip_grads([a], limit)
    assert abs(float(mn.grad_norm([a, a])) - math.sqrt(2) * norm64([a])) < 1e-5  # twice in a norm is fine


def test_repeats_bitwise_graph_and_stream():
    announce("clip", "captured, on another stream")
    grads = [randn(n, seed=i, dtype=[BF16, FP32][i % 2]) for i, n in enumerate([40_000, 17, 1_000_003])]
    out = [torch.zeros_like(g) for g in grads]
    ref_norm = mn.clip_grads(grads, 3.0, out=out).clone()
    ref = [o.clone() for o in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        n2 = mn.clip_grads(grads, 3.0, out=out)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(n2, ref_norm) and all(torch.equal(o, r) for o, r in zip(out, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n3 = mn.clip_grads(grads, 3.0, out=out)
    for scale in (1.0, 2.0, 0.25):
        for g in grads:
            g.mul_(scale)
        graph.replay()
        torch.cuda.synchronize()
        got_norm, got = n3.clone(), [o.clone() for o in out]
        eager = mn.clip_grads(grads, 3.0, out=out)
        assert torch.equal(eager, got_norm) and all(torch.equal(o, r) for o, r in zip(out, got))
    # two graphs may run at once: each has its own scratch
    assert torch.equal(mn.grad_norm(grads), mn.grad_norm(grads, workspace=mn.Workspace()))


def test_clip_then_step():
    """The clipped gradients are those that a step of scaled gradients takes."""
    announce("clip", "in front of a step")
    shapes = [(256, 128), (128, 384)]
    grads = [randn(r * c, seed=i).view(r, c) for i, (r, c) in enumerate(shapes)]
    ps, qs = ([randn(r * c, seed=9 + i).view(r, c) for i, (r, c) in enumerate(shapes)] for _ in range(2))
    bs, cs = ([torch.zeros_like(g) for g in grads] for _ in range(2))
    norm = float(mn.grad_norm(grads))
    c = torch.tensor(float(torch.tensor(1.0, dtype=torch.float64) / (norm64(grads) + float(torch.tensor(1e-6)))),
                     dtype=FP32, device=DEV)
    scaled = [g * c for g in grads]
    mn.clip_grads(grads, 1.0)
    assert norm > 1.0 and all(torch.equal(a, b) for a, b in zip(grads, scaled))
    mn.step(ps, grads, bs, mu=0.95, lr=0.02)
    mn.step(qs, scaled, cs, mu=0.95, lr=0.02)
    assert all(torch.equal(a, b) for a, b in zip(ps + bs, qs + cs))
