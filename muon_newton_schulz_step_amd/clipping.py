"""The norm of a model's gradients and their clipping, in front of a Muon step.
Argument marshalling only: the kernels are behind ``include/muon.h``.

    norm = clip_grads(grads, 1.0)          # in place
    step(params, grads, bufs, mu=0.95, lr=0.02)

``grads`` may mix matrices and vectors, bf16 and fp32; each is contiguous (a view
into a flat buffer may begin at any element).  Nothing here waits for the GPU:
the norm comes back as a tensor.
"""
from __future__ import annotations

import ctypes

from . import _workspace_tensor, lib
from . import layers as _layers


def _tensors(ts, name: str, index):
    """(pointers, element counts, dtype codes, device index) of a list of tensors."""
    codes = _layers._codes
    try:
        kinds = [codes[t.dtype] for t in ts]
    except KeyError as e:
        raise TypeError(f"{name}: unsupported dtype {e.args[0]} (bfloat16 or float32)") from None
    for t in ts:
        if not t.is_contiguous():
            raise ValueError(f"{name}: every tensor must be contiguous")
        if t.get_device() != index:
            raise ValueError(f"{name}: every tensor must be on one GPU, found {t.device}")
    return [t.data_ptr() for t in ts], [t.numel() for t in ts], kinds


def _array(ctype, values):
    return (ctype * max(1, len(values)))(*values)


def _prepare(grads, workspace, out=None):
    """What both entry points hand on: (device index, new norm, workspace bytes, arguments)."""
    torch = _layers._torch()
    grads = list(grads)
    if not grads:
        raise ValueError("grads must hold at least one tensor")
    index = _layers._device(grads[0], _workspace_tensor(workspace))
    ptrs, counts, kinds = _tensors(grads, "grads", index)
    sizes = _array(ctypes.c_longlong, counts)
    args = [len(ptrs), sizes, _array(ctypes.c_void_p, ptrs), _array(ctypes.c_int, kinds)]
    if out is not None:
        out = list(out)
        optrs, ocounts, okinds = _tensors(out, "out", index)
        if len(out) != len(grads) or any(o.shape != g.shape for o, g in zip(out, grads)):
            raise ValueError("out must hold a tensor of each gradient's shape")
        args += [_array(ctypes.c_void_p, optrs), _array(ctypes.c_int, okinds)]
    norm = torch.empty((), dtype=torch.float32, device=grads[0].device)
    return index, norm, lib().muon_grad_norm_workspace_bytes(len(ptrs), sizes), args


def grad_norm(grads, *, workspace=None):
    """The norm of all gradients together, sqrt(sum of squares), as an fp32
    tensor without dimensions.  Summed in 64 bits."""
    index, norm, need, args = _prepare(grads, workspace)
    _layers._call_with_scratch(index, "muon_grad_norm", need, workspace, *args, norm.data_ptr())
    return norm


def clip_grads(grads, max_norm: float, *, eps: float = 1e-6, out=None, workspace=None):
    """Scales the gradients by max_norm / (norm + eps) where that is below 1, in
    place or into ``out`` (tensors of the same shapes, bf16 or fp32: fp32
    accumulators can be clipped into the bf16 gradients of a step).  Returns the
    norm before clipping, as ``grad_norm`` does.  A norm that is infinite or NaN
    takes the gradients with it, as the formula says."""
    index, norm, need, args = _prepare(grads, workspace, out)
    if out is None:
        args += [None, None]
    _layers._call_with_scratch(index, "muon_clip_grads", need, workspace, *args, max_norm, eps,
                               norm.data_ptr())
    return norm
