"""The operators of a block together, as a training step uses them: norm, MLP in 8
bits with squared ReLU, gated residual sum and the next norm, a loss, all the way
back, the gradients' norm, clipping and the Muon step, against the same step in 64
bits on the values that the 8-bit operands stand for, eager and captured."""
import numpy as np
import pytest
import torch

import muon_newton_schulz_step_amd as mn
from gpu_helpers import announce, to64
from oracle import layers_oracle as lo

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def randn(*shape, seed=0, std=1.0, mean=0.0):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV) * std + mean


def values(t):
    q = to64(t.data.float())[:, :t.cols]
    e = t.scale.cpu().numpy().astype(np.int64)[:, :-(-t.cols // 128)] - 127
    return q * lo.expand(e, q.shape, t.block_rows)


class Block:
    def __init__(self, tokens, d, ff, rms):
        self.rms = rms
        self.up, self.down = randn(ff, d, seed=1, std=d ** -0.5), randn(d, ff, seed=2, std=ff ** -0.5)
        self.bup, self.bdown = randn(ff, seed=3, std=0.1), randn(d, seed=4, std=0.1)
        self.g1, self.g2, self.pg = (randn(d, seed=s, std=0.1, mean=1.0) for s in (5, 6, 7))
        self.gate, self.scale = randn(d, seed=8, std=0.1, mean=0.5), torch.full((1,), 0.9, device=DEV)
        self.x = randn(tokens, d, seed=9)
        self.dr, self.dh = randn(tokens, d, seed=10, std=0.1), randn(tokens, d, seed=11, std=0.1).to(BF16)
        self.bufs = [torch.zeros_like(self.up), torch.zeros_like(self.down)]

    def forward(self):
        self.up8, self.up8t = mn.quantize8(self.up, 128, transposed=True)
        self.down8, self.down8t = mn.quantize8(self.down, 128, transposed=True)
        _, self.h8, self.s1 = mn.residual_norm(self.x, None, self.g1, rms=self.rms, out_dtype=E4M3)
        self.a8, self.z = mn.linear8(self.h8, self.up8, self.bup, activation="relu2", keep=True, out_dtype=E4M3)
        self.y = mn.linear8(self.a8, self.down8, self.bdown)
        self.r, self.h, self.s2 = mn.residual_norm(self.x, self.y, self.g2, post_weight=self.pg, gate=self.gate,
                                                   scale=self.scale, rms=self.rms, out_dtype=BF16)

    def backward(self):
        self.b2 = mn.residual_norm_backward(self.dr, self.dh, self.r, self.y, self.g2, self.s2, x=self.x, bias=False,
                                            post_weight=self.pg, gate=self.gate, scale=self.scale, rms=self.rms)
        dy, self.dy8, self.dbdown = mn.linear8_backward(self.b2.dbranch)
        self.ddown = mn.weight_grad(dy, self.a8)
        self.dz, self.dz8, self.dbup = mn.linear8_backward(mn.matmul8(self.dy8, self.down8t), self.z, activation="relu2")
        self.dup = mn.weight_grad(self.dz, self.h8)
        dh1 = mn.matmul8(self.dz8, self.up8t, out_dtype=FP32)
        self.b1 = mn.residual_norm_backward(self.b2.dx, dh1, self.x, None, self.g1, self.s1, bias=False, rms=self.rms)

    def grads(self):
        return [self.dup, self.ddown, self.dbup, self.dbdown, self.b1.dweight, self.b2.dweight,
                self.b2.dpost_weight, self.b2.dgate, self.b2.dscale]

    def step(self, max_norm):
        self.norm = mn.clip_grads(self.grads(), max_norm)
        mn.step([self.up, self.down], [self.dup, self.ddown], self.bufs, mu=0.95, lr=0.02)


def close(got, ref, tol, what):
    err = np.linalg.norm(to64(got.float()) - ref) / np.linalg.norm(ref)
    assert err <= tol, (what, err)


@pytest.mark.parametrize("tokens,d,ff,rms", [(200, 256, 640, True), (77, 384, 1003, False), (1, 128, 512, True)])
def test_block(tokens, d, ff, rms):
    """Relative errors in the 2-norm.  A rounding to bf16 is uniform within half a
    step, 2^-9 relative in the root mean square at most, one to 8 bits 2^-5; what
    follows a gradient in 8 bits (the weight gradient's operands are bf16 dz and the
    8-bit activation, which the reference takes as it is) has one of those: 2^-5 of
    its terms, and twice that is allowed for the sums."""
    announce("block", tokens, d, ff, rms)
    b = Block(tokens, d, ff, rms)
    b.forward()
    x, up, down = to64(b.x), values(b.up8), values(b.down8)
    _, h, s1 = lo.residual_norm(x, None, to64(b.g1), rms=rms)
    close(b.h8.dequantize(), h, 2.0 ** -5, "h8")
    y1, z = lo.linear8(values(b.h8), up, to64(b.bup), "relu2", None)
    close(b.z, z, 2.0 ** -8, "z")
    close(b.a8.dequantize(), y1, 2.0 ** -5, "a8")
    y, _ = lo.linear8(values(b.a8), down, to64(b.bdown), None, None)
    close(b.y, y, 2.0 ** -8, "y")
    o = dict(pw=to64(b.pg), gate=to64(b.gate), scale=to64(b.scale), rms=rms)
    r, h2, s2 = lo.residual_norm(x, to64(b.y), to64(b.g2), **o)
    close(b.r, r, 1e-5, "r")
    close(b.h, h2, 2.0 ** -8, "h")
    b.backward()
    ref = lo.residual_norm_backward(to64(b.dr), to64(b.dh), r, to64(b.y), to64(b.g2), s2, x, **o)
    for name in ("dx", "dweight", "dpost_weight", "dgate", "dscale"):
        close(getattr(b.b2, name), np.atleast_1d(ref[name]), 1e-4, name)
    dy = ref["dbranch"]
    close(b.b2.dbranch, dy, 2.0 ** -8, "dbranch")
    close(b.dbdown, dy.sum(0), 2.0 ** -7, "dbdown")
    close(b.ddown, dy.T @ values(b.a8), 2.0 ** -7, "ddown")
    da = dy @ down
    dz = da * lo.activation_grad(z, "relu2")
    close(b.dz, dz, 2.0 ** -4, "dz")
    close(b.dup, dz.T @ values(b.h8), 2.0 ** -4, "dup")
    dx1 = lo.residual_norm_backward(ref["dx"], dz @ up, x, None, to64(b.g1), s1, rms=rms)
    close(b.b1.dx, dx1["dx"], 2.0 ** -3, "dx of the block")
    before = [t.clone() for t in (b.up, b.down)]
    grads = [to64(g) for g in b.grads()]
    norm = np.sqrt(sum((g ** 2).sum() for g in grads))
    b.step(0.5 * norm)
    assert abs(float(b.norm) - norm) <= 1e-6 * norm
    for got, g in zip(b.grads(), grads):
        assert np.allclose(to64(got), g * 0.5 * norm / (norm + 1e-6), rtol=1e-6, atol=0)
    for w, w0 in zip((b.up, b.down), before):
        assert torch.isfinite(w).all() and not torch.equal(w, w0)


def test_block_captured():
    """The whole of it in one graph, replayed on new inputs, with eager work between."""
    announce("block captured")
    b, e = Block(150, 256, 640, True), Block(150, 256, 640, True)

    def run(k):
        k.forward()
        k.backward()
        k.step(1.0)
        return [k.r, k.h, k.norm, *k.grads(), k.b1.dx, k.up, k.down, *k.bufs]

    run(b)  # (workspaces, library streams)
    run(e)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(b)
    for seed in (21, 22, 23):
        b.x.copy_(randn(150, 256, seed=seed))
        e.x.copy_(b.x)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        ref = run(e)
        assert all(torch.equal(p, q) for p, q in zip(kept, ref))
