"""linear8's choice of exact products without a GPU: its flag in the C ABI, and that the
operands of tests/test_gpu_linear8_exact.py tell exact products from cut ones."""
import numpy as np

import muon_newton_schulz_step_amd as mn
from test_linear8_cpu import INVALID, OK, P, forward, t8


def test_flag():
    exact = mn.MUON_EXACT
    for act in range(6):
        assert forward(act=act | exact, a=t8(1, 0)) == OK
    assert forward(act=6 | exact) == forward(act=exact << 1) == forward(act=-exact) == INVALID
    assert forward(act=exact, y=P) == INVALID                     # its other checks stay


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
