"""The gradients' norm and clipping without a GPU: sizes and refusals of the C
ABI (every rejected call returns before any HIP call is made) and the binding's
checks."""
import ctypes

import pytest
import torch

import muon_newton_schulz_step_amd as mn

P = 0x100000  # aligned, never dereferenced by rejected calls
INVALID, WORKSPACE = mn.MUON_ERR_INVALID_ARG, mn.MUON_ERR_WORKSPACE
BF16, FP32 = mn.MUON_BF16, mn.MUON_FP32
TILE, GROUPS, TENSORS = 16384, 2048, 128


def arr(ctype, v):
    return None if v is None else (ctype * max(1, len(v)))(*v)


def call(clip, n=None, sizes=(100, 7), grads=(P, P + 4096), dtypes=(BF16, FP32), out=None,
         out_dtypes=None, max_norm=1.0, eps=1e-6, norm=P * 2, ws=P * 3, ws_bytes=1 << 16):
    n = len(sizes) if n is None else n
    common = (n, arr(ctypes.c_longlong, sizes), arr(ctypes.c_void_p, grads), arr(ctypes.c_int, dtypes))
    if clip:
        return mn.lib().muon_clip_grads(*common, arr(ctypes.c_void_p, out), arr(ctypes.c_int, out_dtypes),
                                        max_norm, eps, norm, ws, ws_bytes, None)
    return mn.lib().muon_grad_norm(*common, norm, ws, ws_bytes, None)


@pytest.mark.parametrize("clip", [False, True])
@pytest.mark.parametrize("kw,expect", [
    (dict(n=-1), INVALID), (dict(n=(1 << 20) + 1), INVALID), (dict(sizes=None, n=2), INVALID),
    (dict(grads=None), INVALID), (dict(dtypes=None), INVALID), (dict(dtypes=(BF16, 2)), INVALID),
    (dict(sizes=(100, -1)), INVALID), (dict(sizes=((1 << 38) + 1, 1)), INVALID),
    (dict(grads=(0, P)), INVALID), (dict(grads=(P + 1, P + 4096)), INVALID),
    (dict(grads=(P, P + 4098)), INVALID),                      # fp32 at half a number
    (dict(norm=0), INVALID), (dict(norm=P * 2 + 2), INVALID),
    (dict(norm=P + 196), INVALID),                             # overlaps a gradient
    (dict(ws=0), WORKSPACE), (dict(ws=P * 3 + 8), WORKSPACE), (dict(ws_bytes=15), WORKSPACE),
    (dict(ws=P), INVALID), (dict(norm=P * 3 + 4), INVALID),    # overlap the workspace
])
def test_refusals(clip, kw, expect):
    assert call(clip, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(max_norm=-1.0), INVALID), (dict(max_norm=float("inf")), INVALID),
    (dict(max_norm=float("nan")), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(out=(P * 4, P * 5)), INVALID),                       # no types
    (dict(out=(P * 4, P * 5), out_dtypes=(BF16, 7)), INVALID),
    (dict(out=(P * 4, 0), out_dtypes=(BF16, BF16)), INVALID),
    (dict(out=(P * 4 + 1, P * 5), out_dtypes=(BF16, BF16)), INVALID),
    (dict(out=(P * 4, P * 4 + 198), out_dtypes=(BF16, BF16)), INVALID),  # overlap each other
    (dict(out=(P, P * 5), out_dtypes=(FP32, BF16)), INVALID),  # in place, but of another type
    (dict(out=(P + 2, P * 5), out_dtypes=(BF16, BF16)), INVALID),
    (dict(out=(P + 4096, P), out_dtypes=(FP32, BF16)), INVALID),  # exchanged
    (dict(grads=(P, P), dtypes=(BF16, BF16)), INVALID),        # scaled twice
])
def test_clip_refusals(kw, expect):
    assert call(True, **kw) == expect


@pytest.mark.parametrize("sizes,parts", [
    ([], 0), ([0, 0], 0), ([1], 1), ([TILE], 1), ([TILE + 1], 2), ([1, 0, 1], 2),
    ([TILE * GROUPS], GROUPS), ([1 << 38], GROUPS), ([1] * TENSORS, TENSORS),
    ([1] * (TENSORS + 1), TENSORS + 1), ([1 << 30] * (TENSORS + 1), 2 * GROUPS),
    ([0] * 500 + [1], 1), ([-1], 0), ([(1 << 38) + 1], 0),
])
def test_workspace(sizes, parts):
    assert mn.lib().muon_grad_norm_workspace_bytes(len(sizes), arr(ctypes.c_longlong, sizes)) == 8 * parts


def test_binding():
    cpu = torch.zeros(4, 4)
    for f in (mn.grad_norm, lambda g, **kw: mn.clip_grads(g, 1.0, **kw)):
        with pytest.raises(ValueError):
            f([])
        with pytest.raises(ValueError):
            f([cpu])
