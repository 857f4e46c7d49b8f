"""ctypes bindings of the operators around the update: layer norm, 8-bit
products with block scales, and orthogonalising stacks of matrices.

Like the rest of the binding these calls check and marshal arguments; the work
is in the library's CUDA kernels.  Each call runs on the device of its tensors,
on `stream` or that device's current stream.  A given stream is also the one
that results and scratch are allocated on, as under `torch.cuda.stream(stream)`.

No call records an autograd graph: results of tensors that require gradients do
not, and the backward calls are the program's own.  A write to `out` counts as an
in-place change, so a graph that saved the tensor refuses its backward pass.

The smallest calls are bound by the host, so the usual case (the current stream
of the current device) takes no context manager and no Stream object.
"""
from __future__ import annotations

import ctypes

from .muonh import (DTYPE_BF16, DTYPE_F16, DTYPE_F32, QUINTIC, BlockOperand, OrthogonalizeDesc, _check, library)

torch = None    # imported by the first call: building the library imports this package without it
_TYPES = {}     # {torch dtype: MUONH_DTYPE_*}


def _types():
    global torch
    if torch is None:
        import torch as module
        _TYPES.update({module.float32: DTYPE_F32, module.bfloat16: DTYPE_BF16, module.float16: DTYPE_F16})
        torch = module
    return _TYPES


def _tensor(t, what: str, dtypes, device=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in dtypes:
        raise TypeError(f"{what} must be a CUDA tensor of dtype {', '.join(map(str, dtypes))}")
    if device is not None and t.device != device:
        raise ValueError(f"{what} must be on {device}, like the other tensors")


def _here(t, stream):
    """The handle of the current stream where the call belongs there; None where it has to move first."""
    index = t.get_device()
    if stream is None and torch._C._cuda_getDevice() == index:
        return torch._C._cuda_getCurrentRawStream(index)
    return None


def _elsewhere(device, stream, call, *args, **kw):
    """`call` with `device` and `stream` as the current ones."""
    if stream is not None and stream.device != device:
        raise ValueError(f"stream must belong to {device}, like the tensors")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        return call(*args, **kw)


def _rows(t, what: str):
    """(pointer, rows, n, row stride) of a tensor seen as rows of its last
    dimension; ValueError where one stride does not lead from row to row."""
    shape = t.shape
    n = shape[-1]
    if t.is_contiguous():
        return t.data_ptr(), (shape[0] if len(shape) == 2 else shape[:-1].numel()), n, n
    if n > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what} must have unit stride in its last dimension")
    rows, ld, expect = 1, None, None
    for size, stride in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):
        rows *= size
        if size == 1:
            continue
        if ld is None:
            ld = stride
        elif stride != expect:
            raise ValueError(f"{what} must be rows one stride apart (call .contiguous())")
        expect = stride * size
    ld = n if ld is None else ld
    if rows > 1 and ld < n:
        raise ValueError(f"{what} must have rows that do not overlap")
    return t.data_ptr(), rows, n, ld


def _like(x):
    """A contiguous tensor of x's shape and type."""
    return torch.empty_like(x) if x.is_contiguous() else torch.empty_like(x, memory_format=torch.contiguous_format)


def _written(out):
    """`out`, whose change autograd is told of."""
    if not out.is_inference():
        torch.autograd.graph.increment_version(out)
    return out


def _vector(t, what: str, n: int, device):
    if t is None:
        return None
    _tensor(t, what, (torch.float32,), device)
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous with {n} elements")
    return t.data_ptr()


def layer_norm(x, weight=None, bias=None, eps=1e-5, rms=False, out=None, stream=None):
    """Layer norm over the last dimension of x (fp32, bf16 or fp16), or the RMS
    norm with rms=True: y = (x - mean) rstd weight + bias.  weight and bias are
    fp32, as adamw_step keeps them.  Returns (y, mean, rstd): y in x's type (or
    `out`, which may be x), mean (None for the RMS norm) and rstd fp32, one per
    row, for layer_norm_backward (no autograd graph is recorded).  The leading
    dimensions of x, and of `out`, have to be rows one stride apart: all heads
    inside a wider projection are two strides and take a .contiguous()."""
    _tensor(x, "x", _types())
    handle = _here(x, stream)
    if handle is None:
        return _elsewhere(x.device, stream, layer_norm, x, weight, bias, eps, rms, out)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must have a last dimension of at least one element")
    device, dtype, lead = x.device, x.dtype, x.shape[:-1]
    xp, rows, n, ldx = _rows(x, "x")
    wp = _vector(weight, "weight", n, device)
    bp = _vector(bias, "bias", n, device)
    given = out is not None
    if not given:
        out = _like(x)
        op, ldo = out.data_ptr(), n
    else:
        _tensor(out, "out", (dtype,), device)
        if out.shape != x.shape:
            raise ValueError("out must have x's shape")
        op, _, _, ldo = _rows(out, "out")
    lead = lead or ((),)   # torch.empty(*sizes) costs half of torch.empty(size)
    mean = None if rms else torch.empty(*lead, dtype=torch.float32, device=device)
    rstd = torch.empty(*lead, dtype=torch.float32, device=device)
    _check(library().muonh_layer_norm(xp, ldx, op, ldo, wp, bp, None if rms else mean.data_ptr(), rstd.data_ptr(),
                                      rows, n, _types()[dtype], eps, handle))
    return _written(out) if given else out, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, bias=False, stream=None):
    """Gradients of layer_norm at x for the gradient dy of its result (x's shape
    and type, rows one stride apart): (dx, dweight, dbias).  mean and rstd are
    what layer_norm gave; mean None means the RMS norm.  dweight (None where
    weight is None) and dbias (None unless bias is true) are fp32, as adamw_step
    reads them, of these rows alone: microbatches' are added by the program."""
    _tensor(x, "x", _types())
    handle = _here(x, stream)
    if handle is None:
        return _elsewhere(x.device, stream, layer_norm_backward, dy, x, weight, mean, rstd, bias)
    device, dtype = x.device, x.dtype
    _tensor(dy, "dy", (dtype,), device)
    if x.dim() < 1 or x.shape[-1] < 1 or dy.shape != x.shape:
        raise ValueError("dy and x must have the same shape, with a last dimension of at least one element")
    xp, rows, n, ldx = _rows(x, "x")
    dyp, _, _, lddy = _rows(dy, "dy")
    wp = _vector(weight, "weight", n, device)
    mp = _vector(mean, "mean", rows, device)
    rp = _vector(rstd, "rstd", rows, device)
    if rp is None:
        raise TypeError("rstd must be given")
    lib = library()
    dx = _like(x)
    dweight = None if weight is None else torch.empty_like(weight)
    dbias = torch.empty(n, dtype=torch.float32, device=device) if bias else None
    size = lib.muonh_layer_norm_workspace(rows, n) if weight is not None or bias else 0
    work = torch.empty(size, dtype=torch.uint8, device=device) if size else None
    _check(lib.muonh_layer_norm_backward(
        dyp, lddy, xp, ldx, wp, mp, rp, dx.data_ptr(), n, None if dweight is None else dweight.data_ptr(),
        None if dbias is None else dbias.data_ptr(), rows, n, _types()[dtype],
        None if work is None else work.data_ptr(), size, handle))
    return dx, dweight, dbias


def _stack(t, what: str):
    """(pointer, matrix stride, row stride) of a 2-D or 3-D tensor as a stack of matrices."""
    shape, strides = t.shape, t.stride()
    rows, cols = shape[-2], shape[-1]
    if cols > 1 and strides[-1] != 1:
        raise ValueError(f"{what} must have unit column stride")
    if rows > 1 and strides[-2] < cols:
        raise ValueError(f"{what} must have rows that do not overlap")
    return t.data_ptr(), strides[0] if len(shape) == 3 else 0, max(strides[-2], cols)


def _apart(batch, rows, cols, stride, ld):
    """Whether no element of a stack with these strides (ld >= cols) belongs to two of its matrices."""
    height = (rows - 1) * ld + cols
    if batch < 2 or stride >= height:                                  # one behind the other
        return True
    if stride < cols or ld >= (batch - 1) * stride + cols:             # side by side in their rows
        return stride >= cols
    for shift in range(stride, min((batch - 1) * stride, height) + 1, stride):   # rows of one between another's
        row, col = divmod(shift, ld)
        if (row < rows and col < cols) or (row + 1 < rows and ld - col < cols):
            return False
    return True


def orthogonalize(x, *, ns_steps=5, ns_coeffs=QUINTIC, eps=1e-7, out=None, stream=None):
    """The Newton-Schulz output of each matrix of a stack x ([rows, cols] or
    [batch, rows, cols], bf16 or fp16, unit column stride, any other strides),
    for matrices whose smaller side is at most 128: one Muon update per
    attention head (an fp32 momentum is cast first).  Returns a tensor of x's shape and type, laid out like x
    where x has no gaps, or `out`, which may be x.  Runs whose factors grow
    beyond 512 (more than five of the default steps) are computed in fp64, and
    take longer."""
    _types()
    _tensor(x, "x", (torch.bfloat16, torch.float16))
    handle = _here(x, stream)
    if handle is None:
        return _elsewhere(x.device, stream, orthogonalize, x, ns_steps=ns_steps, ns_coeffs=ns_coeffs, eps=eps, out=out)
    shape = x.shape
    if len(shape) not in (2, 3):
        raise ValueError("x must be a matrix or a stack of matrices")
    xp, xs, ldx = _stack(x, "x")
    a, b, c = ns_coeffs
    batch = shape[0] if len(shape) == 3 else 1
    rows, cols = shape[-2], shape[-1]
    lib = library()
    given = out is not None
    if not given:
        # matrices that overlap along a row have no layout of their own to keep
        out = torch.empty_like(x) if batch < 2 or xs >= cols else torch.empty(shape, dtype=x.dtype, device=x.device)
    else:
        _tensor(out, "out", (x.dtype,), x.device)
        if out.shape != shape:
            raise ValueError("out must have x's shape")
    op, os_, ldo = _stack(out, "out")
    if not _apart(batch, rows, cols, os_, ldo):
        raise ValueError("out must have matrices that do not overlap")
    d = OrthogonalizeDesc(xp, op, batch, rows, cols, xs, ldx, os_, ldo, _types()[x.dtype], int(ns_steps), a, b, c, eps)
    size = lib.muonh_orthogonalize_workspace(ctypes.byref(d))
    work = torch.empty(size, dtype=torch.uint8, device=x.device) if size else None
    _check(lib.muonh_orthogonalize(ctypes.byref(d), None if work is None else work.data_ptr(), size, handle))
    return _written(out) if given else out


def _matrix(t, what: str):
    """(pointer, rows, cols, row stride) of a 2-D tensor with unit column stride."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{what} must be 2-D")
    rows, cols = shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{what} must have unit column stride")
    if rows > 1 and ld < cols:
        raise ValueError(f"{what} must have rows that do not overlap")
    return t.data_ptr(), rows, cols, ld if ld > cols else cols


def _quantize(x, block_rows, rows, columns, stream):
    _tensor(x, "x", _types())
    handle = _here(x, stream)
    if handle is None:
        return _elsewhere(x.device, stream, _quantize, x, block_rows, rows, columns, None)
    device = x.device
    xp, m, n, ldx = _matrix(x, "x")
    out = []

    def room(r, c):
        """r x c bytes with a row stride that is a multiple of 16, and their scales."""
        ld, groups = -(-c // 16) * 16, -(-c // 128)
        q = torch.empty(r, ld, dtype=torch.float8_e4m3fn, device=device)
        s = torch.empty(-(-r // block_rows), groups, dtype=torch.uint8, device=device)
        out.append(q if ld == c else q[:, :c])
        out.append(s)
        return q.data_ptr(), ld, s.data_ptr(), groups

    args = room(m, n) if rows else (None, 0, None, 0)
    args += room(n, m) if columns else (None, 0, None, 0)
    _check(library().muonh_block_quantize(xp, ldx, m, n, _types()[x.dtype], block_rows, *args, handle))
    return tuple(out)


def block_quantize(x, rows=True, columns=False, stream=None):
    """x [m, n] (fp32, bf16 or fp16) in e4m3 with a power-of-two scale for each
    1 x 128 group: (q, scale) along its rows, and with columns=True also (qt,
    scale_t), its transpose in groups along x's columns (the weight gradient's
    operand).  q is float8_e4m3fn with a row stride that is a multiple of 16,
    scale is uint8 [m, ceil(n / 128)], the exponent plus 127."""
    if not rows and not columns:
        raise ValueError("rows or columns must be true")
    return _quantize(x, 1, rows, columns, stream)


def block_quantize_weight(w, stream=None):
    """w [n, k] in e4m3 with a scale for each 128 x 128 block, and its transpose:
    (q, scale, qt, scale_t), for the forward product and the activation gradient."""
    return _quantize(w, 128, True, True, stream)


def _block_operand(q, scale, what: str, device=None):
    _types()
    _tensor(q, what, (torch.float8_e4m3fn,), device)
    _tensor(scale, f"{what}_scale", (torch.uint8,), q.device)
    qp, rows, k, ld = _matrix(q, what)
    sp, srows, groups, lds = _matrix(scale, f"{what}_scale")
    if groups != -(-k // 128) or (srows != rows and srows != -(-rows // 128)):
        raise ValueError(f"{what}_scale must be [{rows} or {-(-rows // 128)}, {-(-k // 128)}] for {what} [{rows}, {k}]")
    return BlockOperand(qp, sp, rows, ld, lds, 1 if srows == rows else 128, 0), rows, k


def block_matmul(a, a_scale, b, b_scale, *, dtype=None, out=None, accumulate=False, stream=None):
    """a b^T for operands of block_quantize or block_quantize_weight: a [m, k]
    and b [n, k] in float8_e4m3fn with uint8 scales for each row or each 128
    rows, and each 128 columns.  Returns [m, n] in dtype (bf16 by default; fp32
    or fp16) or writes to `out`; accumulate=True adds to an fp32 `out`, such as
    the gradient that MuonH.step reads."""
    ao, m, k = _block_operand(a, a_scale, "a")
    handle = _here(a, stream)
    if handle is None:
        return _elsewhere(a.device, stream, block_matmul, a, a_scale, b, b_scale, dtype=dtype, out=out,
                          accumulate=accumulate)
    bo, n, kb = _block_operand(b, b_scale, "b", a.device)
    if k != kb:
        raise ValueError("a and b must have the same number of columns")
    given = out is not None
    if not given:
        if accumulate:
            raise ValueError("accumulate needs out")
        dtype = torch.bfloat16 if dtype is None else dtype
        if dtype not in _types():
            raise TypeError("dtype must be torch.float32, torch.bfloat16 or torch.float16")
        out = torch.empty(m, n, dtype=dtype, device=a.device)
        op, ldo = out.data_ptr(), n
    else:
        _tensor(out, "out", _types() if dtype is None else (dtype,), a.device)
        if out.shape != (m, n):
            raise ValueError(f"out must be [{m}, {n}]")
        op, _, _, ldo = _matrix(out, "out")
    _check(library().muonh_block_matmul(ctypes.byref(ao), ctypes.byref(bo), k, op, ldo, _types()[out.dtype],
                                        1 if accumulate else 0, handle))
    return _written(out) if given else out


def operator_status(stream=None) -> None:
    """Synchronises `stream` (default: the current one) and raises MuonHError if
    a device wait gave up in an operator call on its device since the previous
    check.  There is one record per device, which reading clears: it holds for
    the calls of all threads and streams, and the first to ask gets it."""
    _types()
    if stream is None:
        stream = torch.cuda.current_stream()
    with torch.cuda.device(stream.device):
        _check(library().muonh_operator_status(stream.cuda_stream))
