"""What stands between a block and the next one: the block's output, normed or
not, gated and added to the scaled residual stream, and the norm in front of the
next block.  Argument marshalling only: the kernels are behind ``include/muon.h``.

    r, h8, stats = residual_norm(x, y, g, post_weight=pg, gate=gate, rms=True,
                                 out_dtype=torch.float8_e4m3fn)
    a8, z = linear8(h8, up8, activation="relu2", keep=True, out_dtype=torch.float8_e4m3fn)
    y = linear8(a8, down8)                                   # the next branch
    ...                                                      # dr, dy
    dz, dz8, _ = linear8_backward(matmul8(quantize8(dy), down8t), z, activation="relu2")
    dh = matmul8(dz8, up8t)
    back = residual_norm_backward(dr, dh, r, y, g, stats, post_weight=pg, gate=gate, rms=True,
                                  bias=False)

The backward passes are calls of their own: autograd records none of these.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

from . import _lib, _workspace_tensor, lib
from . import layers as _layers
from .layers import (MUON_BF16, Tensor8, _call, _call_with_scratch, _device, _dtype_code, _matrix,
                     _vector, _within_int)


class ResidualNormGrads(NamedTuple):
    """Gradients of residual_norm's operands and parameters; None where there is none."""
    dx: object
    dbranch: object
    dweight: object
    dbias: object
    dpost_weight: object
    dpost_bias: object
    dgate: object
    dscale: object


def _params(cols, weight, bias, post_weight, post_bias, gate, scale, rms, eps):
    if post_bias is not None and post_weight is None:
        raise ValueError("post_bias needs post_weight")
    vectors = (("weight", weight, cols), ("bias", bias, cols), ("post_weight", post_weight, cols),
               ("post_bias", post_bias, cols), ("gate", gate, cols), ("scale", scale, 1))
    ptrs = [None if v is None else _vector(v, n, name) for name, v, n in vectors]
    return _lib.MuonResidualParams(*ptrs, eps, 1 if rms else 0)


def residual_norm(x, branch, weight, bias=None, *, post_weight=None, post_bias=None, gate=None,
                  scale=None, rms: bool = False, eps: float = 1e-5, out_dtype=None):
    """(r, h, stats) of the residual stream ``x`` and a block's output ``branch``,
    (rows, cols) both:

        p = norm(branch) * post_weight + post_bias     (without post_weight: branch)
        r = scale * x + gate * p
        h = norm(r) * weight + bias

    with layer norms, or RMS norms (``rms``).  ``weight``, ``bias``, ``post_weight``,
    ``post_bias`` and ``gate`` are fp32 vectors, ``scale`` an fp32 tensor of one
    element; all but ``weight`` may be None.  ``branch`` None: the norm in front of
    the first block, r = scale * x.  r has x's dtype; h is ``out_dtype``, bf16 or
    fp32 (default: branch's), or torch.float8_e4m3fn for a Tensor8 with blocks of
    1 x 128.  ``stats`` (4, rows) is for the backward pass.  Everything is fp32 up to
    the one rounding of each result; h comes from r before that."""
    torch = _layers._torch()
    xp, rows, cols, ldx = _matrix(x, "x")
    code = bcode = _dtype_code(x.dtype)
    bp, ldb = None, cols
    if branch is not None:
        if branch.shape != (rows, cols):
            raise ValueError("branch must have x's shape")
        bp, _, _, ldb = _matrix(branch, "branch")
        bcode = _dtype_code(branch.dtype)
    elif post_weight is not None or gate is not None:
        raise ValueError("post_weight and gate need a branch")
    p = _params(cols, weight, bias, post_weight, post_bias, gate, scale, rms, eps)
    index = _device(x, branch, weight, bias, post_weight, post_bias, gate, scale)
    device = x.device
    if branch is None and scale is None:
        r, rp = x, None
    else:
        r = torch.empty(rows, cols, dtype=x.dtype, device=device)
        rp = r.data_ptr()
    out_dtype = out_dtype or (x if branch is None else branch).dtype
    if out_dtype == torch.float8_e4m3fn:
        h = Tensor8.empty(rows, cols, 1, device)
        hp, hcode, h8 = None, MUON_BF16, h._c
    else:
        hcode = _dtype_code(out_dtype)
        h = torch.empty(rows, cols, dtype=out_dtype, device=device)
        hp, h8 = h.data_ptr(), None
    stats = torch.empty(4, rows, dtype=torch.float32, device=device)
    _call(index, "muon_residual_norm", xp, code, ldx, bp, bcode, ldb, rows, cols, p, rp, cols, hp,
          hcode, cols, h8, stats.data_ptr())
    return r, h, stats


def residual_norm_backward_workspace_bytes(rows: int, cols: int, branch_params: bool) -> int:
    """Bytes of residual_norm_backward's workspace, ``branch_params`` where it has a
    post_weight or a gate; 0 also for sizes that it refuses."""
    if not _within_int(rows, cols):
        return 0
    return int(lib().muon_residual_norm_backward_workspace_bytes(rows, cols, 1 if branch_params else 0))


def residual_norm_backward(dr, dh, r, branch, weight, stats, *, x=None, bias: bool = True,
                           post_weight=None, post_bias=None, gate=None, scale=None,
                           rms: bool = False, into=None, accumulate: bool = False, workspace=None):
    """The gradients of residual_norm, a ResidualNormGrads, from those of its
    results: ``dr`` (x's dtype; None: none) and ``dh`` (branch's dtype).  ``r``,
    ``stats`` and the parameters are the forward pass's; ``branch`` None where it was
    None there; ``x`` is needed with a ``scale``.  ``bias`` False: no dbias.
    dx has x's dtype, dbranch branch's; where they are the same numbers of the
    same dtype (no post_weight, gate and scale) they are one tensor.  ``into``: a
    ResidualNormGrads whose parameter gradients (fp32) are written, or with
    ``accumulate`` added to; what it has of dx and dbranch is not used."""
    torch = _layers._torch()
    rp, rows, cols, ldr = _matrix(r, "r")
    code = _dtype_code(r.dtype)
    dhp, drows, dcols, lddh = _matrix(dh, "dh")
    bcode = _dtype_code(dh.dtype)
    if (drows, dcols) != (rows, cols):
        raise ValueError("dh must have r's shape")
    if stats.dtype != torch.float32 or stats.shape != (4, rows) or not stats.is_contiguous():
        raise ValueError("stats must be the forward pass's (4, rows)")

    def operand(t, name, dtype):
        if t is None:
            return None, cols
        if t.shape != (rows, cols) or t.dtype != dtype:
            raise ValueError(f"{name} must have r's shape and be of {dtype}")
        ptr, _, _, ld = _matrix(t, name)
        return ptr, ld

    drp, lddr = operand(dr, "dr", r.dtype)
    of_branch = post_weight is not None or gate is not None
    if of_branch and branch is None:
        raise ValueError("post_weight and gate need a branch")
    bp, ldb = operand(branch, "branch", dh.dtype)
    if scale is not None and x is None:
        raise ValueError("scale needs x")
    xp, ldx = operand(x if scale is not None else None, "x", r.dtype)
    p = _params(cols, weight, None, post_weight, post_bias, gate, scale, rms, 0.0)
    if accumulate and into is None:
        raise ValueError("accumulate needs into")
    index = _device(r, dr, dh, branch, weight, stats, post_weight, post_bias, gate, scale,
                    x if scale is not None else None, _workspace_tensor(workspace),
                    *(into[2:] if into is not None else ()))
    device = r.device
    wanted = (("dweight", True, cols), ("dbias", bias, cols), ("dpost_weight", post_weight is not None, cols),
              ("dpost_bias", post_bias is not None, cols), ("dgate", gate is not None, cols),
              ("dscale", scale is not None, 1))
    grads, ptrs = [], []
    for k, (name, there, n) in enumerate(wanted):
        given = into[2 + k] if into is not None else None
        if not there:
            if given is not None:
                raise ValueError(f"into has {name}, of a parameter that is not there")
            grads.append(None)
            ptrs.append(None)
            continue
        if given is None:
            if accumulate:
                raise ValueError(f"accumulate needs {name} in into")
            given = torch.empty(n, dtype=torch.float32, device=device)
            ptrs.append(given.data_ptr())
        else:
            ptrs.append(_vector(given, n, name))
        grads.append(given)
    dx = torch.empty(rows, cols, dtype=r.dtype, device=device)
    if branch is None:
        db = dbp = None
    elif not of_branch and scale is None and bcode == code:
        db, dbp = dx, None
    else:
        db = torch.empty(rows, cols, dtype=dh.dtype, device=device)
        dbp = db.data_ptr()
    need = lib().muon_residual_norm_backward_workspace_bytes(rows, cols, 1 if of_branch else 0)
    _call_with_scratch(index, "muon_residual_norm_backward", need, workspace, drp, lddr, dhp, lddh, rp,
                       ldr, bp if of_branch else None, ldb, xp, ldx, code, bcode, rows, cols, p,
                       stats.data_ptr(), dx.data_ptr(), cols, dbp, cols,
                       ctypes.byref(_lib.MuonResidualGrads(*ptrs)), 1 if accumulate else 0)
    return ResidualNormGrads(dx, db, *grads)
