"""The norm of a model's gradients and their clipping, in front of a Muon step.
Argument marshalling only: the kernels are behind ``include/muon.h``.

    norm = clip_grads(grads, 1.0)          # in place
    step(params, grads, bufs, mu=0.95, lr=0.02)

``grads`` may mix matrices and vectors, bf16 and fp32; each is contiguous (a view
into a flat buffer may begin at any element).  Nothing here waits for the GPU:
the norm comes back as a tensor.
"""
from __future__ import annotations

from array import array
from operator import attrgetter

from . import _workspace_tensor, lib
from . import layers as _layers

_dtype, _shape = attrgetter("dtype"), attrgetter("shape")


def _tensors(ts, name: str, index: int):
    """(pointers, element counts, dtype codes) of a list of tensors, as arrays.  What is
    asked of each tensor is asked of all of them at once: a model has hundreds, and
    the GPU is done with a small one's in 20 us."""
    cls = _layers._T.Tensor
    kinds = list(map(_layers._codes.get, map(_dtype, ts)))
    if None in kinds:
        raise TypeError(f"{name}: unsupported dtype {ts[kinds.index(None)].dtype} (bfloat16 or float32)")
    if not all(map(cls.is_contiguous, ts)):
        raise ValueError(f"{name}: every tensor must be contiguous")
    if set(map(cls.get_device, ts)) != {index}:
        raise ValueError(f"{name}: every tensor must be on cuda:{index}")
    return array("Q", map(cls.data_ptr, ts)), array("q", map(cls.numel, ts)), array("i", kinds)


def _prepare(grads, workspace, out=None):
    """What both entry points hand on: (device index, new norm, workspace bytes,
    arguments, and the arrays that they point to)."""
    torch = _layers._torch()
    grads = list(grads)
    if not grads:
        raise ValueError("grads must hold at least one tensor")
    index = _layers._device(grads[0], _workspace_tensor(workspace))
    kept = list(_tensors(grads, "grads", index))
    if out is not None:
        out = list(out)
        if list(map(_shape, out)) != list(map(_shape, grads)):
            raise ValueError("out must hold a tensor of each gradient's shape")
        optrs, _, okinds = _tensors(out, "out", index)
        kept += [optrs, okinds]
    ptrs, sizes, *rest = (a.buffer_info()[0] for a in kept)
    norm = torch.empty((), dtype=torch.float32, device=grads[0].device)
    need = lib().muon_grad_norm_workspace_bytes(len(grads), sizes)
    return index, norm, need, [len(grads), sizes, ptrs, *rest], kept


def grad_norm(grads, *, workspace=None):
    """The norm of all gradients together, sqrt(sum of squares), as an fp32
    tensor without dimensions.  Summed in 64 bits."""
    index, norm, need, args, kept = _prepare(grads, workspace)
    _layers._call_with_scratch(index, "muon_grad_norm", need, workspace, *args, norm.data_ptr())
    del kept  # until the launches
    return norm


def clip_grads(grads, max_norm: float, *, eps: float = 1e-6, out=None, workspace=None):
    """Scales the gradients by max_norm / (norm + eps) where that is below 1, in
    place or into ``out`` (tensors of the same shapes, bf16 or fp32: fp32
    accumulators can be clipped into the bf16 gradients of a step).  Returns the
    norm before clipping, as ``grad_norm`` does.  A norm that is infinite or NaN
    takes the gradients with it, as the formula says."""
    index, norm, need, args, kept = _prepare(grads, workspace, out)
    if out is None:
        args += [None, None]
    _layers._call_with_scratch(index, "muon_clip_grads", need, workspace, *args, max_norm, eps,
                               norm.data_ptr())
    del kept
    return norm
