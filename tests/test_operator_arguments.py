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
