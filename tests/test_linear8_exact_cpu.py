"""linear8's choice of products without a GPU: its flags in the C ABI, and that the operands
of tests/test_gpu_linear8_exact.py tell exact products from cut ones."""
import numpy as np
import pytest

import muon_newton_schulz_step_amd as mn
from test_linear8_cpu import INVALID, OK, P, forward, t8


def test_flags():
    exact, fast = mn.MUON_EXACT, mn.MUON_FAST
    for act in range(6):
        assert forward(act=act | exact, a=t8(1, 0)) == forward(act=act | fast, a=t8(1, 0)) == OK
        assert forward(act=act | exact, dtype=mn.MUON_FP32, a=t8(1, 0)) == OK
        assert forward(act=act | fast, dtype=mn.MUON_FP32, a=t8(1, 0)) == INVALID
        assert forward(act=act | fast | exact, a=t8(1, 0)) == INVALID
    y8 = t8(3, 0, 16)
    assert forward(act=fast, dtype=mn.MUON_FP32, y=0, y8=y8, a=t8(1, 0)) == OK
    assert forward(act=6 | exact) == forward(act=6 | fast) == forward(act=fast << 1) == INVALID
    assert forward(act=-exact) == forward(act=-fast) == forward(act=exact - 1) == INVALID
    assert forward(act=exact, y=P) == forward(act=fast, y=P) == INVALID  # its other checks stay


def test_binding_refusals():
    a, b = mn.Tensor8.empty(8, 256, device="cpu"), mn.Tensor8.empty(16, 256, 128, device="cpu")
    for exact in (True, False, None):
        with pytest.raises(ValueError):            # not on a GPU
            mn.linear8(a, b, exact=exact)


def cut(a, b):
    """A planted mistake: sums of products cut 13 bits below the largest of their group of 8."""
    k = -(-a.shape[1] // 8) * 8
    p = a[:, None, :] * b[None]
    p = np.pad(p, ((0, 0), (0, 0), (0, k - a.shape[1]))).reshape(*p.shape[:2], -1, 8)
    top = np.abs(p).max(-1, keepdims=True)
    unit = 2.0 ** (np.floor(np.log2(np.maximum(top, 1.0))) - 13)
    return (np.trunc(p / unit) * unit).sum((-1, -2))


def test_operands_show_a_cut():
    rng = np.random.default_rng(0)
    a, b = rng.integers(-2, 3, (6, 300)) * 1.0, rng.integers(-2, 3, (7, 300)) * 1.0
    assert np.array_equal(cut(a, b), a @ b.T)                     # small whole numbers do not
    for c in range(3, 268, 64):
        sign = rng.integers(0, 2, 7) * 2.0 - 1.0
        a[:, c], a[:, c + 32], b[:, c], b[:, c + 32] = 256.0, 256.0, 256.0 * sign, -256.0 * sign
    assert (cut(a, b) != a @ b.T).mean() > 0.9
