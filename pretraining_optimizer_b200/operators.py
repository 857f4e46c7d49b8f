"""ctypes bindings of the operators around the update: layer norm, 8-bit
products with block scales, and orthogonalising stacks of matrices.

Like the rest of the binding these calls check and marshal arguments; the work
is in the library's CUDA kernels.  Each call runs on the device of its tensors,
on `stream` or that device's current stream.  A given stream is also the one
that results and scratch are allocated on, as under `torch.cuda.stream(stream)`.
"""
from __future__ import annotations

import contextlib
import ctypes

from .muonh import DTYPE_BF16, DTYPE_F16, DTYPE_F32, QUINTIC, BlockOperand, OrthogonalizeDesc, _check, library


def _dtype_code(dtype):
    import torch
    codes = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}
    return codes.get(dtype)


def _tensor(t, what: str, dtypes, device=None):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in dtypes:
        raise TypeError(f"{what} must be a CUDA tensor of dtype {', '.join(map(str, dtypes))}")
    if device is not None and t.device != device:
        raise ValueError(f"{what} must be on {device}, like the other tensors")
    return t


@contextlib.contextmanager
def _on_other(device, stream):
    import torch
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream().cuda_stream
        else:
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


def _on(device, stream):
    """Context in which a call's allocations and launches belong to `device` and
    `stream`; gives the stream's handle."""
    import torch
    if stream is None and torch.cuda.current_device() == device.index:
        return contextlib.nullcontext(torch.cuda.current_stream().cuda_stream)
    return _on_other(device, stream)


def _rows(t, what: str):
    """(pointer, rows, n, row stride) of a tensor seen as rows of its last
    dimension; ValueError where one stride does not lead from row to row."""
    n = t.shape[-1]
    rows = 1
    for d in t.shape[:-1]:
        rows *= d
    if t.is_contiguous():
        return t.data_ptr(), rows, n, n
    if n > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what} must have unit stride in its last dimension")
    ld, expect = None, None
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
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


def _vector(t, what: str, n: int, device):
    import torch
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
    row, for layer_norm_backward."""
    import torch
    _tensor(x, "x", (torch.float32, torch.bfloat16, torch.float16))
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must have a last dimension of at least one element")
    xp, rows, n, ldx = _rows(x, "x")
    wp = _vector(weight, "weight", n, x.device)
    bp = _vector(bias, "bias", n, x.device)
    with _on(x.device, stream) as handle:
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        _tensor(out, "out", (x.dtype,), x.device)
        if out.shape != x.shape:
            raise ValueError("out must have x's shape")
        op, _, _, ldo = _rows(out, "out")
        mean = None if rms else torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        _check(library().muonh_layer_norm(xp, ldx, op, ldo, wp, bp, None if rms else mean.data_ptr(),
                                          rstd.data_ptr(), rows, n, _dtype_code(x.dtype), eps, handle))
    return out, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, bias=False, stream=None):
    """Gradients of layer_norm at x for the gradient dy of its result (x's shape
    and type): (dx, dweight, dbias).  mean and rstd are what layer_norm gave;
    mean None means the RMS norm.  dweight (None where weight is None) and dbias
    (None unless bias is true) are fp32, as adamw_step reads them."""
    import torch
    _tensor(x, "x", (torch.float32, torch.bfloat16, torch.float16))
    _tensor(dy, "dy", (x.dtype,), x.device)
    if x.dim() < 1 or x.shape[-1] < 1 or dy.shape != x.shape:
        raise ValueError("dy and x must have the same shape, with a last dimension of at least one element")
    xp, rows, n, ldx = _rows(x, "x")
    dyp, _, _, lddy = _rows(dy, "dy")
    wp = _vector(weight, "weight", n, x.device)
    mp = _vector(mean, "mean", rows, x.device)
    rp = _vector(rstd, "rstd", rows, x.device)
    if rp is None:
        raise TypeError("rstd must be given")
    lib = library()
    with _on(x.device, stream) as handle:
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dweight = None if weight is None else torch.empty(weight.shape, dtype=torch.float32, device=x.device)
        dbias = torch.empty(n, dtype=torch.float32, device=x.device) if bias else None
        size = lib.muonh_layer_norm_workspace(rows, n) if weight is not None or bias else 0
        work = torch.empty(size, dtype=torch.uint8, device=x.device) if size else None
        _check(lib.muonh_layer_norm_backward(
            dyp, lddy, xp, ldx, wp, mp, rp, dx.data_ptr(), n, None if dweight is None else dweight.data_ptr(),
            None if dbias is None else dbias.data_ptr(), rows, n, _dtype_code(x.dtype),
            None if work is None else work.data_ptr(), size, handle))
    return dx, dweight, dbias


def _stack(t, what: str):
    """(pointer, matrix stride, row stride) of a 2-D or 3-D tensor as a stack of matrices."""
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what} must have unit column stride")
    if t.shape[-2] > 1 and t.stride(-2) < t.shape[-1]:
        raise ValueError(f"{what} must have rows that do not overlap")
    return t.data_ptr(), t.stride(0) if t.dim() == 3 else 0, max(t.stride(-2), t.shape[-1])


def orthogonalize(x, *, ns_steps=5, ns_coeffs=QUINTIC, eps=1e-7, out=None, stream=None):
    """The Newton-Schulz output of each matrix of a stack x ([rows, cols] or
    [batch, rows, cols], bf16 or fp16, unit column stride, any other strides),
    for matrices whose smaller side is at most 128: one Muon update per
    attention head.  Returns a tensor of x's shape and type, or `out`, which
    may be x."""
    import torch
    _tensor(x, "x", (torch.bfloat16, torch.float16))
    if x.dim() not in (2, 3):
        raise ValueError("x must be a matrix or a stack of matrices")
    xp, xs, ldx = _stack(x, "x")
    a, b, c = ns_coeffs
    rows, cols = x.shape[-2:]
    lib = library()
    with _on(x.device, stream) as handle:
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        _tensor(out, "out", (x.dtype,), x.device)
        if out.shape != x.shape:
            raise ValueError("out must have x's shape")
        op, os_, ldo = _stack(out, "out")
        if x.dim() == 3 and x.shape[0] > 1 and os_ < cols:
            raise ValueError("out must have matrices that do not overlap")
        d = OrthogonalizeDesc(xp, op, x.shape[0] if x.dim() == 3 else 1, rows, cols, xs, ldx, os_, ldo,
                              _dtype_code(x.dtype), int(ns_steps), a, b, c, eps)
        size = lib.muonh_orthogonalize_workspace(ctypes.byref(d))
        work = torch.empty(size, dtype=torch.uint8, device=x.device) if size else None
        _check(lib.muonh_orthogonalize(ctypes.byref(d), None if work is None else work.data_ptr(), size, handle))
    return out


def _matrix(t, what: str):
    """(pointer, rows, cols, row stride) of a 2-D tensor with unit column stride."""
    if t.dim() != 2:
        raise ValueError(f"{what} must be 2-D")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{what} must have unit column stride")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{what} must have rows that do not overlap")
    return t.data_ptr(), t.shape[0], t.shape[1], max(t.stride(0), t.shape[1])


def _quantize(x, block_rows, rows, columns, stream):
    import torch
    _tensor(x, "x", (torch.float32, torch.bfloat16, torch.float16))
    xp, m, n, ldx = _matrix(x, "x")
    out = []

    def room(r, c):
        """r x c bytes with a row stride that is a multiple of 16, and their scales."""
        ld, groups = -(-c // 16) * 16, -(-c // 128)
        q = torch.empty((r, ld), dtype=torch.float8_e4m3fn, device=x.device)
        s = torch.empty((-(-r // block_rows), groups), dtype=torch.uint8, device=x.device)
        out.extend((q if ld == c else q[:, :c], s))
        return q.data_ptr(), ld, s.data_ptr(), groups

    with _on(x.device, stream) as handle:
        args = room(m, n) if rows else (None, 0, None, 0)
        args += room(n, m) if columns else (None, 0, None, 0)
        _check(library().muonh_block_quantize(xp, ldx, m, n, _dtype_code(x.dtype), block_rows, *args, handle))
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


def _block_operand(q, scale, what: str, device):
    import torch
    _tensor(q, what, (torch.float8_e4m3fn,), device)
    _tensor(scale, f"{what}_scale", (torch.uint8,), device)
    qp, rows, k, ld = _matrix(q, what)
    sp, srows, groups, lds = _matrix(scale, f"{what}_scale")
    if groups != -(-k // 128) or srows not in (rows, -(-rows // 128)):
        raise ValueError(f"{what}_scale must be [{rows} or {-(-rows // 128)}, {-(-k // 128)}] for {what} [{rows}, {k}]")
    return BlockOperand(qp, sp, rows, ld, lds, 1 if srows == rows else 128, 0), rows, k


def block_matmul(a, a_scale, b, b_scale, *, dtype=None, out=None, accumulate=False, stream=None):
    """a b^T for operands of block_quantize or block_quantize_weight: a [m, k]
    and b [n, k] in float8_e4m3fn with uint8 scales for each row or each 128
    rows, and each 128 columns.  Returns [m, n] in dtype (bf16 by default; fp32
    or fp16) or writes to `out`; accumulate=True adds to an fp32 `out`, such as
    the gradient that MuonH.step reads."""
    import torch
    ao, m, k = _block_operand(a, a_scale, "a", None)
    bo, n, kb = _block_operand(b, b_scale, "b", a.device)
    _tensor(a_scale, "a_scale", (torch.uint8,), a.device)
    if k != kb:
        raise ValueError("a and b must have the same number of columns")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        dtype = torch.bfloat16 if dtype is None else dtype
    elif dtype is not None and dtype != out.dtype:
        raise ValueError("out must be of dtype")
    with _on(a.device, stream) as handle:
        if out is None:
            if _dtype_code(dtype) is None:
                raise TypeError("dtype must be torch.float32, torch.bfloat16 or torch.float16")
            out = torch.empty((m, n), dtype=dtype, device=a.device)
        _tensor(out, "out", (torch.float32, torch.bfloat16, torch.float16), a.device)
        if out.shape != (m, n):
            raise ValueError(f"out must be [{m}, {n}]")
        op, _, _, ldo = _matrix(out, "out")
        _check(library().muonh_block_matmul(ctypes.byref(ao), ctypes.byref(bo), k, op, ldo, _dtype_code(out.dtype),
                                            int(bool(accumulate)), handle))
    return out


def operator_status(stream=None) -> None:
    """Synchronises `stream` (default: the current one) and raises MuonHError
    if a device wait gave up in an operator call since the previous check."""
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    _check(library().muonh_operator_status(stream.cuda_stream))
