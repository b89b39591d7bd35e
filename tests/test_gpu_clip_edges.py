"""Clipping to a limit of zero without eps, and of many tensors at once."""
import pytest
import torch

import muon_newton_schulz_step_amd as mn
from gpu_helpers import announce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_zeros_without_eps(dtype):
    """0 / 0 is not below 1: the gradients, all zeros, stay as they are."""
    announce("clip: zeros, a limit of zero, no eps", dtype)
    g = torch.zeros(40_000, dtype=dtype, device=DEV)
    g[7] = -0.0
    kept, out = g.clone(), torch.full_like(g, 5.0)
    for limit in (0.0, 1.0):
        assert float(mn.clip_grads([g], limit, eps=0.0, out=[out])) == 0.0
        assert torch.equal(out, kept)
        assert float(mn.clip_grads([g], limit, eps=0.0)) == 0.0
        assert torch.equal(g, kept)
    g[3] = 2.0                                                # and a limit of zero is still one
    assert float(mn.clip_grads([g], 0.0, eps=0.0)) == 2.0 and (g == 0).all()


def kernels_ms(f):
    """The least time of a call's kernels, from the timing log."""
    times = []
    for _ in range(6):
        mn.timing_read()
        mn.timing_enable(True)
        try:
            f()
            torch.cuda.synchronize()
            (r,) = mn.timing_read()
        finally:
            mn.timing_enable(False)
        times.append(r["ms"])
    return min(times)


def many(count, size):
    flat = torch.zeros(count * size, dtype=BF16, device=DEV)
    flat[::size] = 1.0
    return flat, list(flat.split(size))


def test_many_tensors():
    """Launches of 128 tensors each: the norm, clipped results and repeats."""
    announce("clip: 1500 tensors")
    flat, grads = many(1500, 20_001)
    kept = flat.clone()
    norm = mn.clip_grads(grads, 1.0)
    assert float(norm) == float(mn.grad_norm(list(kept.split(20_001)))) == float(torch.tensor(1500.0).sqrt())
    c = torch.tensor(1.0 / (1500.0 ** 0.5 + 1e-6), dtype=torch.float64).to(FP32)
    assert torch.equal(flat, (kept.float() * c).to(BF16))
    again = kept.clone()
    assert torch.equal(mn.clip_grads(list(again.split(20_001)), 1.0), norm) and torch.equal(again, flat)
    out = torch.zeros_like(kept)
    assert torch.equal(mn.clip_grads(list(kept.split(20_001)), 1.0, out=list(out.split(20_001))), norm)
    assert torch.equal(out, flat)


def test_work_grows_with_the_tensors():
    """Gradients that stay as they are cost the clipping pass next to nothing, however many
    launches there are: at most as much again as their norm."""
    announce("clip: 4000 tensors of 262144")
    _, grads = many(4000, 1 << 18)
    norm, clip = kernels_ms(lambda: mn.grad_norm(grads)), kernels_ms(lambda: mn.clip_grads(grads, 1e6))
    print("norm", norm, "ms, clip", clip, "ms")
    assert clip <= 2.5 * norm


def test_many_tensors_captured():
    announce("clip: 1500 tensors, captured")
    flat, grads = many(1500, 20_001)
    out = torch.zeros_like(flat)
    outs = list(out.split(20_001))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = mn.clip_grads(grads, 1.0, out=outs)
    for k in (2.0, 0.25, 8.0):
        flat.mul_(k)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got, clipped = norm.clone(), out.clone()
        assert torch.equal(mn.clip_grads(grads, 1.0, out=outs), got) and torch.equal(out, clipped)
        assert float(got) == float(mn.grad_norm(grads))
