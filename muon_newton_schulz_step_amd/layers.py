"""Linear layers in 8 bits and layer norm: what the stepped matrices are used
for between two Muon steps.  Argument marshalling only, as in the package's
``__init__``: every computation is a HIP kernel behind ``include/muon.h``.

One linear layer y = x W^T behind a layer norm, forward and backward, and the
step of its weights:

    h8, mean, rstd = layer_norm(x, g, b, out_dtype=torch.float8_e4m3fn)
    w8, w8t = quantize8(W, block_rows=128, transposed=True)   # once per step
    y = matmul8(h8, w8)
    ...                                                       # dy
    dh = matmul8(quantize8(dy), w8t)
    dx, dg, db = layer_norm_backward(dh, x, g, mean, rstd)
    dW = weight_grad(dy, h8)                 # or out=dW, accumulate=True
    step([W], [dW], [buf], mu=0.95, lr=0.02)

The backward passes are calls of their own: autograd records none of these.
Matrices may have a row stride, and begin at a multiple of 16 bytes (every new
tensor does; a slice that does not is refused: clone() it first).
"""
from __future__ import annotations

import threading

from . import _lib
from . import (MUON_BF16, MUON_EXACT, MUON_FAST, MUON_FP32, MUON_OK, MuonError, Workspace,
               _workspace_tensor, lib)

_MAX_ROWS = _lib.MUON_MAX_ROWS

# torch, its raw stream and device queries and the element types' codes, from
# the first call on, and the library's functions
_T = None
_stream_of = _current_device = None
_codes: dict = {}
_functions: dict = {}


def _torch():
    global _T, _stream_of, _current_device
    if _T is None:
        import torch
        _codes.update({torch.bfloat16: MUON_BF16, torch.float32: MUON_FP32})
        _stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _T = torch
    return _T


def _dtype_code(dtype) -> int:
    code = _codes.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype} (bfloat16 or float32)")
    return code


def _ld8(cols: int) -> int:
    return -(-cols // 128) * 128


def _scale_ld8(cols: int) -> int:
    return -(-cols // 512) * 4


class Tensor8:
    """A matrix in 8 bits: e4m3 values and a power-of-two scale for each block
    of ``block_rows`` x 128 (1 or 128 rows).

    data   (rows, ld) torch.float8_e4m3fn, ld = cols rounded up to 128, the
           padding columns zero
    scale  (ceil(rows / block_rows), ceil(cols / 512) * 4) torch.uint8: the
           byte e + 127 of the scale 2^e

    A value is its e4m3 number times its block's scale.  The tensors may be
    written in place, but not exchanged for others."""

    # one made by `empty` holds both in one allocation, and makes the two
    # tensors when they are first asked for
    __slots__ = ("_data", "_scale", "_buf", "_index", "_cols", "_block_rows", "_c")

    def __init__(self, data, scale, cols: int, block_rows: int = 1):
        torch = _T or _torch()
        if block_rows not in (1, 128):
            raise ValueError("block_rows must be 1 or 128")
        if not 1 <= cols <= _lib.MUON_MAX_COLS8:
            raise ValueError(f"cols must lie in [1, {_lib.MUON_MAX_COLS8}]")
        if data.dtype != torch.float8_e4m3fn or scale.dtype != torch.uint8:
            raise TypeError("data must be float8_e4m3fn and scale uint8")
        if data.dim() != 2 or data.shape[1] != _ld8(cols) or not data.is_contiguous():
            raise ValueError("data must be contiguous, (rows, cols rounded up to 128)")
        rows = data.shape[0]
        if rows > _lib.MUON_MAX_ROWS:
            raise ValueError(f"at most {_lib.MUON_MAX_ROWS} rows")
        if scale.shape != (-(-rows // block_rows), _scale_ld8(cols)) or not scale.is_contiguous():
            raise ValueError("scale must be contiguous, (blocks of rows, 4 ceil(cols / 512))")
        index = data.get_device()
        if scale.get_device() != index:
            raise ValueError("data and scale must be on one device")
        self._data, self._scale, self._buf = data, scale, None
        self._index, self._cols, self._block_rows = index, cols, block_rows
        self._c = _lib.MuonTensor8(data.data_ptr(), scale.data_ptr(), rows, cols, block_rows)

    @classmethod
    def empty(cls, rows: int, cols: int, block_rows: int = 1, device=None):
        torch = _T or _torch()
        if (block_rows not in (1, 128) or not 0 <= rows <= _lib.MUON_MAX_ROWS
                or not 1 <= cols <= _lib.MUON_MAX_COLS8):
            raise ValueError("rows in [0, MUON_MAX_ROWS], cols in [1, MUON_MAX_COLS8], "
                             "block_rows 1 or 128")
        t = cls.__new__(cls)
        nbytes = rows * _ld8(cols)
        buf = torch.empty(nbytes + -(-rows // block_rows) * _scale_ld8(cols), dtype=torch.uint8,
                          device=device)
        t._data = t._scale = None
        t._buf, t._index, t._cols, t._block_rows = buf, buf.get_device(), cols, block_rows
        ptr = buf.data_ptr()
        t._c = _lib.MuonTensor8(ptr, ptr + nbytes, rows, cols, block_rows)
        return t

    @property
    def data(self):
        if self._data is None:
            rows, ld = self._c.rows, _ld8(self._cols)
            self._data = self._buf[:rows * ld].view((_T or _torch()).float8_e4m3fn).view(rows, ld)
        return self._data

    @property
    def scale(self):
        if self._scale is None:
            rows = self._c.rows
            self._scale = self._buf[rows * _ld8(self._cols):].view(
                -(-rows // self._block_rows), _scale_ld8(self._cols))
        return self._scale

    @property
    def cols(self) -> int:
        return self._cols

    @property
    def block_rows(self) -> int:
        return self._block_rows

    @property
    def rows(self) -> int:
        return self._c.rows

    @property
    def shape(self):
        return (self._c.rows, self._cols)

    @property
    def device(self):
        return (self._data if self._buf is None else self._buf).device

    def get_device(self) -> int:
        return self._index

    def dequantize(self, dtype=None):
        return dequantize8(self, dtype)

    def __repr__(self):
        return f"Tensor8({self.rows} x {self.cols}, blocks of {self.block_rows} x 128)"


# The checks below run on every call, where a small one takes a few
# microseconds on the GPU: they ask each tensor as little as they can.
def _matrix(t, name: str):
    """(pointer, rows, cols, row stride) of a 2-D tensor whose rows are dense."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = t.shape
    if cols < 1:
        raise ValueError(f"{name} must have at least one column")
    if rows > _MAX_ROWS or cols > _MAX_ROWS:  # the C ABI's sizes are 32-bit
        raise ValueError(f"{name} has more than {_MAX_ROWS} rows or columns")
    ld, inner = t.stride()
    if (inner != 1 and cols > 1) or (ld < cols and rows > 1):
        raise ValueError(f"{name}: elements of a row must be adjacent, and rows not overlap "
                         "(an expanded or transposed tensor: contiguous() first)")
    return t.data_ptr(), rows, cols, ld if rows > 1 else cols


def _vector(t, n: int, name: str):
    if t.dtype != (_T or _torch()).float32 or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 vector of {n} elements")
    return t.data_ptr()


def _device(first, *others) -> int:
    """The index of the GPU that every tensor or Tensor8 (None: none) is on."""
    index = first.get_device()
    if index < 0:
        raise ValueError("tensors must be GPU tensors")
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"every tensor must be on cuda:{index}, found {t.device}")
    return index


# The default workspaces of the calls here, one per (device, stream).  A call
# that has one is two launches, which another thread's on the same stream (a
# backward pass runs in a thread of its own) must not come between: it holds the
# lock from before it takes the workspace until both are enqueued.
_workspaces: dict = {}
_lock = threading.Lock()


def _scratch(nbytes: int, index: int, workspace):
    """(pointer, bytes, what keeps it) of the workspace.  The default one of a
    stream is used there only, so that nothing has to be recorded when it is
    large enough.  A call that is being captured takes its own from the graph's
    memory instead: graphs captured on one stream may be replayed on several."""
    torch = _T or _torch()
    if workspace is None:
        if _current_device() == index:
            capturing = torch.cuda.is_current_stream_capturing()
        else:
            with torch.cuda.device(index):
                capturing = torch.cuda.is_current_stream_capturing()
        if capturing:
            buf = torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", index))
            return buf.data_ptr(), nbytes, buf
        key = (index, _stream_of(index))
        workspace = _workspaces.get(key)
        if workspace is None:
            workspace = _workspaces[key] = Workspace()
        buf = workspace.buf
        if buf is not None and buf.numel() >= nbytes:
            return buf.data_ptr(), buf.numel(), buf
    if isinstance(workspace, Workspace):
        workspace = workspace.get(nbytes, torch.device("cuda", index))
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _call(index: int, name: str, *args):
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(lib(), name)
    if _current_device() == index:
        st = fn(*args, _stream_of(index))
    else:
        with _T.cuda.device(index):
            st = fn(*args, _stream_of(index))
    if st != MUON_OK:
        raise MuonError(st, name)


def _call_with_scratch(index: int, name: str, nbytes: int, workspace, *args):
    if nbytes == 0:
        _call(index, name, *args, 0, 0)
        return
    with _lock:
        ptr, size, kept = _scratch(nbytes, index, workspace)
        _call(index, name, *args, ptr, size)
        del kept  # until the launches


def quantize8(x, block_rows: int = 1, *, transposed: bool = False, out=None):
    """``x`` (rows, cols), bf16 or fp32, as a Tensor8.  With ``transposed``
    (128-row blocks only) returns (Tensor8 of x, Tensor8 of x^T): the same
    values and scales in both layouts, in one pass."""
    _T or _torch()
    xp, rows, cols, ldx = _matrix(x, "x")
    code = _dtype_code(x.dtype)
    if transposed and block_rows != 128:
        raise ValueError("a transposed copy needs block_rows=128")
    if transposed and rows == 0:
        raise ValueError("a tensor without rows has no transposed copy")
    if out is not None and (out.shape != (rows, cols) or out.block_rows != block_rows):
        raise ValueError("out must be a Tensor8 of x's shape and block_rows")
    index = _device(x, out)
    if out is None:
        out = Tensor8.empty(rows, cols, block_rows, x.device)
    other = Tensor8.empty(cols, rows, 128, x.device) if transposed else None
    _call(index, "muon_quantize8", xp, code, rows, cols, ldx, out._c,
          other._c if transposed else None)
    return (out, other) if transposed else out


def dequantize8(t, dtype=None):
    """The values of a Tensor8 as bf16 (default) or fp32, exact in both."""
    torch = _T or _torch()
    dtype = dtype or torch.bfloat16
    code = _dtype_code(dtype)
    index = _device(t)
    y = torch.empty(t.rows, t.cols, dtype=dtype, device=t.device)
    _call(index, "muon_dequantize8", t._c, y.data_ptr(), code, t.cols)
    return y


def matmul8(a, b, *, out_dtype=None, out=None):
    """a b^T of two Tensor8, (m, k) and (n, k) -> (m, n) in bf16 (default) or
    fp32, sums in fp32.  ``out`` may have a row stride.

    bf16 results of more than 16 rows (32 where n < 16384) come from an
    instruction that cuts products off 13 bits below the largest of 8, 1.5e-5 of
    the result's norm; all others from exact products.  A row may differ in its
    last bits with the number of rows beside it."""
    torch = _T or _torch()
    if a.cols != b.cols:
        raise ValueError(f"a and b must have the same number of columns: {a.cols}, {b.cols}")
    index = _device(a, b, out)
    m, n = a.rows, b.rows
    if out is None:
        out = torch.empty(m, n, dtype=out_dtype or torch.bfloat16, device=a.device)
        yp, ldy = out.data_ptr(), max(n, 1)
    else:
        if out.shape != (m, n) or (out_dtype or out.dtype) != out.dtype:
            raise ValueError("out must be (a.rows, b.rows) and of out_dtype")
        yp, _, _, ldy = _matrix(out, "out") if n else (0, m, n, 1)
    _call(index, "muon_matmul8", a._c, b._c, yp, _dtype_code(out.dtype), ldy)
    return out


def _activation(name) -> int:
    code = _lib.ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"unknown activation {name!r} (None, "
                         f"{', '.join(repr(a) for a in _lib.ACTIVATIONS if a)})")
    return code


def linear8(a, b, bias=None, *, activation=None, residual=None, keep: bool = False,
            out_dtype=None, out=None, exact=None):
    """act(a b^T + bias) + residual of two Tensor8, (m, k) and (n, k) -> (m, n) in
    bf16 (default), fp32, or torch.float8_e4m3fn: a Tensor8 with blocks of
    1 x 128, the next product's operand.  ``bias`` is fp32, ``residual`` bf16 or fp32;
    ``activation`` None, "relu", "relu2" (squared), "gelu", "gelu_tanh" or
    "silu".  ``keep`` returns (y, z) with z = a b^T + bias for linear8_backward, in
    y's dtype (bf16 beside a Tensor8).  ``out`` may be given: a matrix in bf16 or fp32,
    which may have a row stride, or a Tensor8; none that overlaps ``residual`` or another
    operand.
    Everything is fp32 up to the one rounding of each result.  Products are exact, but
    for bf16 results of many rows, which are those of matmul8 and cut far below their
    rounding, and for plain ones in 8 bits (without bias, activation, residual and
    ``keep``).  ``exact`` True makes these exact as well; False takes matmul8's for every
    8-bit result, up to 1.7 times as fast, but more of its values close to halfway go to
    their other neighbour (include/muon.h has the figures)."""
    torch = _T or _torch()
    if a.cols != b.cols:
        raise ValueError(f"a and b must have the same number of columns: {a.cols}, {b.cols}")
    act = _activation(activation)
    flags = 0 if exact is None else MUON_EXACT if exact else MUON_FAST
    if keep and not act:
        raise ValueError("keep is for an activation: without one the backward pass needs no z")
    m, n = a.rows, b.rows
    bp = _vector(bias, n, "bias") if bias is not None else None
    index = _device(a, b, bias, residual, out)
    device = a.device
    rp, rcode, ldr = None, MUON_BF16, n
    if residual is not None:
        if residual.shape != (m, n):
            raise ValueError("residual must be (a.rows, b.rows)")
        rcode = _dtype_code(residual.dtype)
        if n:
            rp, _, _, ldr = _matrix(residual, "residual")
    out8 = isinstance(out, Tensor8) or (out is None and out_dtype == torch.float8_e4m3fn)
    if out8:
        if n == 0:
            raise ValueError("an 8-bit result has at least one column")
        if out is None:
            out = Tensor8.empty(m, n, 1, device)
        elif out.shape != (m, n) or out.block_rows != 1 or out_dtype not in (None, torch.float8_e4m3fn):
            raise ValueError("out must be (a.rows, b.rows), with blocks of 1 x 128, and of out_dtype")
        yp, code, ldy, y8 = None, MUON_BF16, n, out._c
    elif out is None:
        out = torch.empty(m, n, dtype=out_dtype or torch.bfloat16, device=device)
        yp, code, ldy, y8 = out.data_ptr(), _dtype_code(out.dtype), max(n, 1), None
    else:
        if out.shape != (m, n) or (out_dtype or out.dtype) != out.dtype:
            raise ValueError("out must be (a.rows, b.rows) and of out_dtype")
        yp, _, _, ldy = _matrix(out, "out") if n else (0, m, n, 1)
        code, y8 = _dtype_code(out.dtype), None
    if flags == MUON_FAST and not out8 and code == MUON_FP32:
        raise ValueError("a result in fp32 comes from exact products")
    z = zp = None
    if keep:
        z = torch.empty(m, n, dtype=torch.bfloat16 if out8 else out.dtype, device=device)
        zp = z.data_ptr()
    _call(index, "muon_linear8", a._c, b._c, bp, act + flags, rp, rcode, ldr, zp, n, yp, code, ldy,
          y8)
    return (out, z) if keep else out


def linear8_backward_workspace_bytes(rows: int, cols: int) -> int:
    """Bytes of linear8_backward's workspace; 0 also for sizes that it refuses."""
    return int(lib().muon_linear8_backward_workspace_bytes(rows, cols)) if _within_int(rows, cols) else 0


def linear8_backward(dy, z=None, *, activation=None, bias: bool = True, dbias=None,
                     accumulate: bool = False, workspace=None):
    """(dz, dz8, dbias) of linear8 from its output gradient ``dy`` (rows, n), bf16 or
    fp32: dz = dy act'(z) in bf16 for weight_grad and as a Tensor8 for the input's
    gradient, matmul8(dz8, w8t), and its sum over the rows.  ``z`` is what linear8
    kept; without an activation it is not needed, and a bf16 ``dy`` is itself dz.
    ``dbias`` (fp32) may be given, and is added to with ``accumulate``; ``bias``
    False: no dbias (None).  The residual's gradient is dy."""
    torch = _T or _torch()
    act = _activation(activation)
    dyp, rows, cols, lddy = _matrix(dy, "dy")
    dcode = _dtype_code(dy.dtype)
    zp, zcode, ldz = None, MUON_BF16, cols
    if act:
        if z is None or z.shape != dy.shape:
            raise ValueError("an activation needs z, of dy's shape")
        zp, _, _, ldz = _matrix(z, "z")
        zcode = _dtype_code(z.dtype)
    if not bias and dbias is not None:
        raise ValueError("dbias was given with bias=False")
    if accumulate and dbias is None:
        raise ValueError("accumulate needs dbias")
    dbp = _vector(dbias, cols, "dbias") if dbias is not None else None
    index = _device(dy, z if act else None, dbias, _workspace_tensor(workspace))
    device = dy.device
    dz8 = Tensor8.empty(rows, cols, 1, device)
    if act or dcode != MUON_BF16:
        dz = torch.empty(rows, cols, dtype=torch.bfloat16, device=device)
        dzp = dz.data_ptr()
    else:
        dz, dzp = dy, None
    if bias and dbias is None:
        dbias = torch.empty(cols, dtype=torch.float32, device=device)
        dbp = dbias.data_ptr()
    need = lib().muon_linear8_backward_workspace_bytes(rows, cols) if bias else 0
    _call_with_scratch(index, "muon_linear8_backward", need, workspace, dyp, dcode, lddy, zp, zcode,
                       ldz, act, rows, cols, dzp, cols, dz8._c, dbp, 1 if accumulate else 0)
    return dz, dz8, dbias


def _within_int(*sizes) -> bool:
    """Whether the C ABI's ints can hold the sizes (ctypes cuts others off)."""
    return all(-2 ** 31 <= v < 2 ** 31 for v in sizes)


def weight_grad_workspace_bytes(tokens: int, n: int, k: int) -> int:
    """Bytes of weight_grad's workspace; 0 also for sizes that it refuses."""
    return int(lib().muon_weight_grad_workspace_bytes(tokens, n, k)) if _within_int(tokens, n, k) else 0


def weight_grad(dy, x, *, out_dtype=None, out=None, accumulate: bool = False, workspace=None):
    """dy^T x: the gradient (n, k) of a linear layer's weights from its output
    gradient ``dy`` (tokens, n), bf16, and its input ``x``, a Tensor8 (tokens,
    k).  fp32 (default) or bf16; ``accumulate`` adds to an fp32 ``out``."""
    torch = _T or _torch()
    dyp, tokens, n, lddy = _matrix(dy, "dy")
    k = x.cols
    if x.rows != tokens:
        raise ValueError(f"dy and x must have the same number of rows: {tokens}, {x.rows}")
    if out is None and accumulate:
        raise ValueError("accumulate needs out")
    if out is not None and (out.shape != (n, k) or (out_dtype or out.dtype) != out.dtype
                            or not out.is_contiguous()):
        raise ValueError("out must be contiguous, (dy columns, x columns), and of out_dtype")
    index = _device(dy, x, out, _workspace_tensor(workspace))
    if out is None:
        out = torch.empty(n, k, dtype=out_dtype or torch.float32, device=dy.device)
    _call_with_scratch(index, "muon_weight_grad", lib().muon_weight_grad_workspace_bytes(tokens, n, k),
                       workspace, dyp, _dtype_code(dy.dtype), lddy, tokens, n, x._c, out.data_ptr(),
                       _dtype_code(out.dtype), 1 if accumulate else 0)
    return out


def layer_norm(x, weight, bias=None, *, eps: float = 1e-5, out_dtype=None):
    """Layer norm over the last axis of ``x`` (rows, cols): (y, mean, rstd).
    ``out_dtype`` bf16 or fp32 (default: x's), or torch.float8_e4m3fn for a
    Tensor8 with blocks of 1 x 128.  ``weight`` and ``bias`` are fp32."""
    torch = _T or _torch()
    xp, rows, cols, ldx = _matrix(x, "x")
    wp = _vector(weight, cols, "weight")
    bp = _vector(bias, cols, "bias") if bias is not None else None
    index = _device(x, weight, bias)
    device = x.device
    mean, rstd = weight.new_empty(rows), weight.new_empty(rows)
    out_dtype = out_dtype or x.dtype
    if out_dtype == torch.float8_e4m3fn:
        y = Tensor8.empty(rows, cols, 1, device)
        yp, code, ldy, y8 = None, MUON_BF16, cols, y._c
    else:
        code = _dtype_code(out_dtype)
        y = torch.empty(rows, cols, dtype=out_dtype, device=device)
        yp, ldy, y8 = y.data_ptr(), cols, None
    _call(index, "muon_layer_norm", xp, _dtype_code(x.dtype), ldx, rows, cols, wp, bp, eps,
          yp, code, ldy, y8, mean.data_ptr(), rstd.data_ptr())
    return y, mean, rstd


def layer_norm_backward_workspace_bytes(rows: int, cols: int) -> int:
    """Bytes of layer_norm_backward's workspace; 0 also for sizes that it refuses."""
    return int(lib().muon_layer_norm_backward_workspace_bytes(rows, cols)) if _within_int(rows, cols) else 0


def layer_norm_backward(dy, x, weight, mean, rstd, *, bias: bool = True, dweight=None,
                        dbias=None, accumulate: bool = False, workspace=None):
    """(dx, dweight, dbias) of layer_norm.  ``x`` is the forward pass's input,
    or the Tensor8 that was kept of it; dx has dy's dtype.  ``dweight`` and
    ``dbias`` (fp32) may be given, and are added to with ``accumulate``;
    ``bias`` False: no dbias (None)."""
    torch = _T or _torch()
    dyp, rows, cols, lddy = _matrix(dy, "dy")
    if isinstance(x, Tensor8):
        same = x.shape == (rows, cols)
        xp, xcode, ldx, x8 = None, MUON_BF16, cols, x._c
    else:
        same = x.shape == dy.shape
        xp, _, _, ldx = _matrix(x, "x")
        xcode, x8 = _dtype_code(x.dtype), None
    if not same:
        raise ValueError("x and dy must have the same shape")
    if not bias and dbias is not None:
        raise ValueError("dbias was given with bias=False")
    if accumulate and (dweight is None or (bias and dbias is None)):
        raise ValueError("accumulate needs dweight and dbias")
    wp = _vector(weight, cols, "weight")
    mp, rp = _vector(mean, rows, "mean"), _vector(rstd, rows, "rstd")
    dwp = _vector(dweight, cols, "dweight") if dweight is not None else 0
    dbp = _vector(dbias, cols, "dbias") if dbias is not None else None
    index = _device(dy, x, weight, mean, rstd, dweight, dbias, _workspace_tensor(workspace))
    device = dy.device
    dx = torch.empty(rows, cols, dtype=dy.dtype, device=device)
    if dweight is None:
        dweight = weight.new_empty(cols)
        dwp = dweight.data_ptr()
    if bias and dbias is None:
        dbias = weight.new_empty(cols)
        dbp = dbias.data_ptr()
    _call_with_scratch(index, "muon_layer_norm_backward",
                       lib().muon_layer_norm_backward_workspace_bytes(rows, cols), workspace, dyp,
                       _dtype_code(dy.dtype), lddy, xp, xcode, ldx, x8, rows, cols, wp, mp, rp,
                       dx.data_ptr(), cols, dwp, dbp, 1 if accumulate else 0)
    return dx, dweight, dbias
