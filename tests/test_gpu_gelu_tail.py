"""GELU of results in fp32, and its slope, to the last digits of the tail they are made of."""
import numpy as np
import pytest
import torch

import muon_newton_schulz_step_amd as mn
from gpu_helpers import announce, to64
from oracle import layers_oracle as lo

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FP32 = torch.float32


def test_gelu_tail():
    """GELU of fp32 results, and its slope, relative to the tail that they are made of.

    u = 2^-24, s the smaller of Phi(z) and Phi(-z).  exp(-z^2 / 2) is exp2 of a product
    of three factors each off by u: relative 3 u z^2 / 2, and 2 u of the instruction.
    The factor beside it: 1 / (1 + 0.3 |z|) is off by 4 u, which counts up to twice in
    the polynomial, whose terms are all below twice their sum, with 9 roundings: 26 u; by
    its fit 3 u.  So s is off by (1.5 z^2 + 31) u of itself, the density phi by (1.5 z^2
    + 5) u; results have two roundings more."""
    announce("GELU's tail")
    u = 2.0 ** -24
    z = torch.linspace(-12.5, 12.5, 20011, device=DEV)
    z64 = to64(z)
    s = lo.ndtr(-np.abs(z64))
    for m in (2, 70):
        a, b = mn.quantize8(torch.zeros(m, 128, device=DEV)), mn.quantize8(torch.zeros(20011, 128, device=DEV), 128)
        got = to64(mn.linear8(a, b, z, activation="gelu", out_dtype=FP32))
        ref = z64 * lo.ndtr(z64)
        bound = (1.5 * z64 ** 2 + 33) * u * np.abs(z64) * s + 2 * u * np.abs(ref)
        off = np.abs(got - ref)
        assert (off <= bound).all(), (m, float(np.nanmax(off / bound)))
    one = torch.ones(1, 20011, device=DEV)
    _, _, db = mn.linear8_backward(one, z.view(1, -1), activation="gelu")
    ref = lo.activation_grad(z64, "gelu")
    phi = np.exp(-z64 ** 2 / 2) / np.sqrt(2 * np.pi)
    bound = (1.5 * z64 ** 2 + 33) * u * s + (1.5 * z64 ** 2 + 9) * u * np.abs(z64) * phi + 3 * u * np.abs(ref)
    off = np.abs(to64(db) - ref)
    assert (off <= bound).all(), float(np.nanmax(off / bound))
