"""The operands of tests/test_gpu_scale_gradient.py tell a sum in 64 bits from lanes' sums in
fp32."""
import numpy as np
import pytest


def cancelling(rows, cols, top, seed=0):
    """(d, x) of odd whole numbers below `top`, whose products sum to 2 x at one element: the
    second half of the rows has the first half's negatives, three columns further on, so
    that no lane's roundings are another one's with the sign turned."""
    rng = np.random.default_rng(seed)
    d, x = (2.0 * rng.integers(0, top // 2, (rows // 2, cols)) + 1.0 for _ in range(2))
    low = d.copy()
    d[rows // 3, cols // 2] += 2.0 if d[rows // 3, cols // 2] + 2.0 < top else -2.0
    if d[rows // 3, cols // 2] < low[rows // 3, cols // 2]:
        d, low = low, d
    return np.concatenate((d, -np.roll(low, 3, 1))), np.concatenate((x, np.roll(x, 3, 1)))


def lanes(d, x, rows_of_a_lane):
    """A planted mistake: lanes of eight columns and some rows whose sums are fp32."""
    p = (d * x).astype(np.float32)
    p = p.reshape(-1, rows_of_a_lane, p.shape[1] // 8, 8).transpose(0, 2, 1, 3)
    p = p.reshape(*p.shape[:2], -1)
    acc = np.zeros(p.shape[:2], np.float32)
    for i in range(p.shape[2]):
        acc += p[:, :, i]
    return float(acc.astype(np.float64).sum())


@pytest.mark.parametrize("rows,cols,each", [(40, 496, 4), (4000, 200, 2), (2000, 1280, 4), (300, 8992, 2)])
def test_operands_show_sums_in_fp32(rows, cols, each):
    d, x = cancelling(rows, cols, 1 << 11)
    exact = 2.0 * x[rows // 3, cols // 2]
    assert float((d * x).sum()) == exact
    assert lanes(d, x, each) != exact
