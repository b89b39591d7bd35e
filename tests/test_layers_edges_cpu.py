"""Edges of the 8-bit linear layer and layer norm that need no GPU."""
import numpy as np
import pytest
import torch

import muon_newton_schulz_step_amd as mn
from oracle import layers_oracle as lo

TOP = 2.0 ** 120
BF16_MAX, FP32_MAX = 255 * TOP, (2 - 2.0 ** -23) * 2.0 ** 127


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("v,q", [
    (FP32_MAX, 240), (-FP32_MAX, -240), (BF16_MAX, 240), (-BF16_MAX, -240), (248 * TOP, 240),
    (247.99 * TOP, 240), (240 * TOP, 240), (232 * TOP, 224), (232.01 * TOP, 240)])
def test_oracle_largest_values_stay_finite(v, q, block_rows):
    # a value of a block with e = 120 is within e4m3's half step, 2^-4 of it,
    # and is a number of fp32 and bf16
    x = np.array([[v, 1.0, FP32_MAX, np.inf, np.nan]])
    got, e = lo.quantize8(x, block_rows)
    assert e[0, 0] == 120 and got[0, 0] == q and got[0, 1] == 0 and np.isnan(got[0, 3:]).all()
    value = got[0, 0] * TOP
    assert np.isfinite(np.float32(value)) and abs(value) <= BF16_MAX
    assert abs(value - v) <= 2.0 ** -4 * abs(v)


@pytest.mark.parametrize("workspace", [
    torch.empty(1, dtype=torch.uint8).expand(1 << 30),              # 2^30 elements, one byte
    torch.empty(1 << 12, dtype=torch.uint8)[::2], torch.empty(64, 64)[:, :32], torch.empty(64, 32).t()])
def test_workspaces_with_gaps_are_refused(workspace):
    # the library would write the gaps, or past the tensor's end
    x, v, t = torch.zeros(4, 256), torch.zeros(256), mn.Tensor8.empty(4, 256)
    one = [torch.zeros(8, 8)], [torch.zeros(8, 8)], [torch.zeros(8, 8)]
    for bad in (lambda: mn.weight_grad(x.bfloat16(), t, workspace=workspace),
                lambda: mn.layer_norm_backward(x, x, v, v[:4], v[:4], workspace=workspace),
                lambda: mn.orthogonalize(x, workspace=workspace),
                lambda: mn.step(*one, mu=0.9, lr=0.1, workspace=workspace),
                lambda: mn.step_ex(*one, mu=0.9, lr=0.1, workspace=workspace)):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            bad()


@pytest.mark.parametrize("past", [2 ** 31, 2 ** 32 + 16384, -2 ** 32 + 16384])
def test_workspace_sizes_past_32_bits(past):
    # 2^32 + 16384 tokens must not pass for 16384, which has partial sums
    assert mn.weight_grad_workspace_bytes(16384, 48, 256) > 0
    assert mn.layer_norm_backward_workspace_bytes(16384, 768) > 0
    assert mn.weight_grad_workspace_bytes(past, 48, 256) == 0
    assert mn.weight_grad_workspace_bytes(16384, 2 ** 32 + 48, 256) == 0
    assert mn.layer_norm_backward_workspace_bytes(past, 768) == 0
    assert mn.layer_norm_backward_workspace_bytes(16384, 2 ** 32 + 768) == 0
