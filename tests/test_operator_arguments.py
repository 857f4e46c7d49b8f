"""Refusals of the operators around the update: argument checks that run before any CUDA call (no GPU)."""
import ctypes

import pytest

import pretraining_optimizer_b200 as P

A = 0x10000   # an address that is never read: every call here is refused


def test_layer_norm_checks():
    f = P.library().muonh_layer_norm
    ok = dict(x=A, ldx=64, y=A, ldy=64, w=A, b=A, mean=A, rstd=A, rows=4, n=64, dtype=1, eps=1e-5, stream=None)

    def call(**kw):
        return f(*{**ok, **kw}.values())

    assert call(rows=-1) == 1 and call(n=0) == 1 and call(n=2 ** 31) == 1
    assert call(dtype=3) == 1 and call(dtype=-1) == 1
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1 and call(eps=float("inf")) == 1
    assert call(x=None) == 1 and call(y=None) == 1 and call(rstd=None) == 1
    assert call(ldx=63) == 1 and call(ldy=0) == 1
    assert call(x=A + 1) == 2 and call(y=A + 1) == 2 and call(w=A + 2) == 2 and call(b=A + 1) == 2
    assert call(mean=A + 2) == 2 and call(rstd=A + 3) == 2 and call(dtype=0, x=A + 2) == 2
    assert call(rows=0, x=None, y=None, rstd=None) == 0
    assert P.library().muonh_last_error() == b""


def test_layer_norm_backward_checks():
    lib = P.library()
    size = lib.muonh_layer_norm_workspace(4, 64)
    assert size == 4 * 64 * 2 * 4 and lib.muonh_layer_norm_workspace(10 ** 6, 64) == 512 * 64 * 2 * 4
    assert lib.muonh_layer_norm_workspace(0, 64) == 0 and lib.muonh_layer_norm_workspace(4, 0) == 0
    ok = dict(dy=A, lddy=64, x=A, ldx=64, w=A, mean=A, rstd=A, dx=A, lddx=64, dw=A, db=A, rows=4, n=64, dtype=1,
              work=A, size=size, stream=None)

    def call(**kw):
        return lib.muonh_layer_norm_backward(*{**ok, **kw}.values())

    assert call(rows=-1) == 1 and call(n=0) == 1 and call(dtype=7) == 1
    for name in ("dy", "x", "rstd", "dx"):
        assert call(**{name: None}) == 1
    for name in ("lddy", "ldx", "lddx"):
        assert call(**{name: 63}) == 1
    assert call(work=None) == 1 and call(size=size - 1) == 1
    assert call(work=A + 2) == 2 and call(dw=A + 1) == 2 and call(db=A + 2) == 2 and call(dy=A + 1) == 2


def test_layer_norm_binding_rejects_cpu_tensors():
    import torch
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        P.layer_norm(x)
    with pytest.raises(TypeError):
        P.layer_norm_backward(x, x, None, None, x[:, 0])
    with pytest.raises(TypeError):
        P.layer_norm([1.0])


def test_row_views():
    """Which strides count as rows one stride apart (the checks need no GPU)."""
    import torch
    from pretraining_optimizer_b200.operators import _rows
    x = torch.zeros(6, 4, 10)
    assert _rows(x, "x")[1:] == (24, 10, 10)
    assert _rows(x[:, :, :8], "x")[1:] == (24, 8, 10)
    assert _rows(x[:, 1, 2:7], "x")[1:] == (6, 5, 40)
    assert _rows(x[3], "x")[1:] == (4, 10, 10) and _rows(x[3, 2], "x")[1:] == (1, 10, 10)
    assert _rows(x[:1, :, :3], "x")[1:] == (4, 3, 10)
    assert _rows(x[:, :, :0], "x")[1:3] == (24, 0)
    for bad in (x[:, :3], x[:, :, ::2], x.transpose(0, 1), x[:1, :1].expand(6, 4, 10), x[0, 0].expand(4, 10)):
        with pytest.raises(ValueError):
            _rows(bad, "x")


def _orth(**kw):
    from pretraining_optimizer_b200.muonh import OrthogonalizeDesc
    ok = dict(x=A, out=A, batch=2, rows=32, cols=64, x_stride=2048, ldx=64, out_stride=2048, ldo=64, dtype=1,
              ns_steps=5, ns_a=3.4445, ns_b=-4.775, ns_c=2.0315, eps=1e-7)
    return OrthogonalizeDesc(*{**ok, **kw}.values())


def test_orthogonalize_checks():
    lib = P.library()

    def call(work=None, size=0, **kw):
        return lib.muonh_orthogonalize(ctypes.byref(_orth(**kw)), work, size, None)

    assert lib.muonh_orthogonalize(None, None, 0, None) == 1
    assert call(batch=-1) == 1 and call(rows=-1) == 1 and call(cols=-1) == 1 and call(batch=2 ** 25) == 1
    assert call(dtype=0) == 1 and call(dtype=9) == 1
    assert call(ns_steps=-1) == 1 and call(ns_steps=17) == 1
    assert call(ns_a=float("nan")) == 1 and call(eps=-1e-9) == 1 and call(eps=float("inf")) == 1
    assert call(rows=129, cols=129, ldx=136, ldo=136) == 6 and b"128" in lib.muonh_last_error()
    assert call(x=None) == 1 and call(out=None) == 1
    assert call(ldx=63) == 1 and call(ldo=8) == 1 and call(x_stride=-8) == 1
    assert call(x=A + 1) == 2
    assert call(batch=0, x=None, out=None) == 0 and call(rows=0) == 0 and call(cols=0) == 0


def test_orthogonalize_workspace():
    lib = P.library()

    def size(**kw):
        return lib.muonh_orthogonalize_workspace(ctypes.byref(_orth(**kw)))

    one = 2 * 32 * 64 * 2
    assert size() == 0 and size(batch=0) == 0
    assert size(x=A + 2) == one and size(ldx=65, x_stride=2080) == one and size(x_stride=2049) == one
    assert size(x_stride=0) == one                          # the same matrix twice
    assert size(ldx=65, ldo=65, x_stride=2080, out_stride=2080) == 2 * one
    assert size(cols=61, ldx=61, x_stride=32 * 61, ldo=64) == one
    assert size(batch=1, x_stride=3) == 0 and size(rows=1, ldx=67, ldo=65) == 0
    assert lib.muonh_orthogonalize_workspace(None) == 0
    d = _orth(x=A + 2)
    assert lib.muonh_orthogonalize(ctypes.byref(d), None, one, None) == 1
    assert lib.muonh_orthogonalize(ctypes.byref(d), A, one - 1, None) == 1
    assert lib.muonh_orthogonalize(ctypes.byref(d), A + 8, one, None) == 2


def test_orthogonalize_layout():
    from pretraining_optimizer_b200.muonh import OrthogonalizeDesc as D
    assert ctypes.sizeof(D) == 96 and D.x_stride.offset == 40 and D.dtype.offset == 72 and D.eps.offset == 92


def test_orthogonalize_binding_rejects():
    import torch
    with pytest.raises(TypeError):
        P.orthogonalize(torch.zeros(4, 8, dtype=torch.bfloat16))
    from pretraining_optimizer_b200.operators import _stack
    x = torch.zeros(3, 6, 10)
    assert _stack(x, "x")[1:] == (60, 10) and _stack(x[:, :, 2:7], "x")[1:] == (60, 10)
    assert _stack(x[1], "x")[1:] == (0, 10) and _stack(x.transpose(0, 1), "x")[1:] == (10, 60)
    for bad in (x.mT, x[:, :, ::2], x[:, :1].expand(3, 6, 10)):
        with pytest.raises(ValueError):
            _stack(bad, "x")


def test_block_quantize_checks():
    f = P.library().muonh_block_quantize
    ok = dict(x=A, ldx=64, rows=4, cols=64, dtype=1, block_rows=1, q=A, ldq=64, s=A, lds=1, qt=A, ldqt=16, st=A,
              ldst=1, stream=None)

    def call(**kw):
        return f(*{**ok, **kw}.values())

    assert call(rows=-1) == 1 and call(cols=-1) == 1 and call(rows=2 ** 24) == 1 and call(cols=2 ** 31) == 1
    assert call(dtype=3) == 1 and call(block_rows=64) == 1
    assert call(x=None) == 1 and call(q=None, qt=None) == 1 and call(s=None) == 1 and call(st=None) == 1
    assert call(ldx=63) == 1 and call(ldq=48) == 1 and call(ldqt=0) == 1 and call(lds=0) == 1 and call(ldst=0) == 1
    assert call(cols=200, ldx=200, ldq=208, lds=1) == 1
    assert call(x=A + 1) == 2 and call(q=A + 8) == 2 and call(ldq=72) == 2 and call(qt=A + 4) == 2 and call(ldqt=20) == 2
    assert call(rows=0, x=None, q=None, qt=None) == 0 and call(cols=0) == 0


def test_block_matmul_checks():
    from pretraining_optimizer_b200.muonh import BlockOperand as Op
    f = P.library().muonh_block_matmul
    assert ctypes.sizeof(Op) == 48 and Op.ld.offset == 24 and Op.block_rows.offset == 40

    def call(a=None, b=None, k=300, d=A, ldd=64, dtype=1, accumulate=0):
        ok = dict(q=A, scale=A, rows=32, ld=304, ld_scale=3, block_rows=1, pad_=0)
        x = Op(*{**ok, **(a or {})}.values())
        y = Op(*{**ok, "rows": 64, **(b or {})}.values())
        return f(ctypes.byref(x), ctypes.byref(y), k, d, ldd, dtype, accumulate, None)

    x = Op()
    assert f(None, ctypes.byref(x), 1, A, 1, 0, 0, None) == 1 and f(ctypes.byref(x), None, 1, A, 1, 0, 0, None) == 1
    for side in ("a", "b"):
        assert call(**{side: dict(rows=-1)}) == 1 and call(**{side: dict(block_rows=2)}) == 1
        assert call(**{side: dict(q=None)}) == 1 and call(**{side: dict(scale=None)}) == 1
        assert call(**{side: dict(ld=288)}) == 1 and call(**{side: dict(ld_scale=2)}) == 1
        assert call(**{side: dict(q=A + 4)}) == 2 and call(**{side: dict(ld=301)}) == 2
        assert call(**{side: dict(rows=0, q=None)}) == 0
    assert call(k=-1) == 1 and call(dtype=4) == 1 and call(dtype=1, accumulate=1) == 1
    assert call(d=None) == 1 and call(ldd=63) == 1 and call(d=A + 1) == 2 and call(dtype=0, d=A + 2) == 2
    assert call(k=0, dtype=0, accumulate=1) == 0


def test_block_binding_rejects():
    import torch
    x = torch.zeros(4, 128)
    with pytest.raises(TypeError):
        P.block_quantize(x)
    with pytest.raises(TypeError):
        P.block_quantize_weight(x)
    with pytest.raises(ValueError):
        P.block_quantize(x, rows=False)
    with pytest.raises(TypeError):
        P.block_matmul(x, x, x, x)
