"""Layer norm and RMS norm, forward and backward, vs fp64 (B200 only).

Tolerances.  u = 2^-24 is half a step of fp32.  A row's sum adds at most 16
terms per thread and then a tree over at most 512 threads (5 shuffles and 16
warps in turn), or, for rows above 8192, n/512 terms per thread: D = 48 + n/512
roundings, so a mean over the row is off by at most D u <|terms|>.  The
statistics' errors reach each output once, next to a handful of roundings of
its own (8 here covers the products, the square root and the division).  The
result is rounded once to its type: half a step, eps/2 relative."""
import numpy as np
import pytest

from oracle import operators as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _t():
    import torch
    return torch


def _dtype(name):
    t = _t()
    return {"fp32": t.float32, "bf16": t.bfloat16, "fp16": t.float16}[name]


def _half_step(dtype):
    return _t().finfo(dtype).eps / 2


def _tiny(dtype):
    """Half the spacing of the smallest values of the type."""
    f = _t().finfo(dtype)
    return f.smallest_normal * f.eps / 2


def _data(rows, n, dtype, seed=0):
    t = _t()
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, n)) * np.exp(rng.standard_normal(n)) + 0.5
    dy = rng.standard_normal((rows, n)) * np.exp(rng.standard_normal((rows, 1)))
    w, b = 1 + 0.2 * rng.standard_normal(n), rng.standard_normal(n)
    to = lambda a, d: t.from_numpy(np.ascontiguousarray(a)).to("cuda:0", d)  # noqa: E731
    return to(x, dtype), to(dy, dtype), to(w, t.float32), to(b, t.float32)


def _np(a):
    return None if a is None else a.double().cpu().numpy()


def check_forward(x, w, b, eps, rms, y, mean, rstd):
    rows, n = x.shape
    xs = _np(x)
    yr, mr, rr = O.layer_norm(xs, _np(w), _np(b), eps, rms)
    depth = 48 + n / 512
    wa = 1.0 if w is None else np.abs(_np(w))
    mean_err = 0.0 if rms else depth * U * np.abs(xs).mean(1)
    # rstd: half the relative error of the mean square, whose terms carry the mean's error
    second = ((xs - mr[:, None]) ** 2).mean(1) + eps
    rstd_rel = 0.5 * (depth + 4) * U + mean_err ** 2 / second + mean_err * U / np.sqrt(second) + 4 * U
    if not rms:
        assert np.all(np.abs(_np(mean) - mr) <= mean_err + U * np.abs(mr))
    assert np.all(np.abs(_np(rstd) - rr) <= rstd_rel * rr)
    unit = np.abs((xs - mr[:, None]) * rr[:, None]) * wa
    tol = unit * (rstd_rel[:, None] + 8 * U) + np.reshape(mean_err * rr, (-1, 1)) * wa
    tol = tol + U * np.abs(xs) * rr[:, None] * wa + U * np.abs(yr)
    tol = tol + _half_step(y.dtype) * (np.abs(yr) + tol) + _tiny(y.dtype)
    assert np.all(np.abs(_np(y) - yr) <= tol)


def check_backward(dy, x, w, mean, rstd, dx, dw, db):
    rows, n = x.shape
    dys, xs, rs = _np(dy), _np(x), _np(rstd)
    rms = mean is None
    ms = np.zeros(rows) if rms else _np(mean)
    dxr, dwr, dbr = O.layer_norm_backward(dys, xs, _np(w), ms, rs, rms)
    xh = (xs - ms[:, None]) * rs[:, None]
    xh_err = 3 * U * (np.abs(xs) + np.abs(ms)[:, None]) * rs[:, None]
    g = np.abs(dys) * (1.0 if w is None else np.abs(_np(w)))
    depth = 48 + n / 512
    mg = 0.0 if rms else (depth + 4) * U * g.mean(1, keepdims=True)
    mgx = (g * np.abs(xh)).mean(1, keepdims=True)
    mgx_err = (depth + 6) * U * mgx + (g * xh_err).mean(1, keepdims=True)
    # the terms themselves are rounded as they are added
    parts = g + (0.0 if rms else g.mean(1, keepdims=True)) + np.abs(xh) * mgx
    tol = rs[:, None] * (6 * U * parts + mg + np.abs(xh) * mgx_err + xh_err * (mgx + mgx_err))
    tol = tol + _half_step(dx.dtype) * (np.abs(dxr) + tol) + _tiny(dx.dtype)
    assert np.all(np.abs(_np(dx) - dxr) <= tol)
    # down the rows: a group's rows in turn (at most rows, at least 1/148/2 of them per block), then 64 groups,
    # 32 partial rows in turn and 16 slices
    down = rows / min(rows, 64) + 64 + 32 + 16 + 4
    if dw is not None:
        assert np.all(np.abs(_np(dw) - dwr) <= (down * U * np.abs(dys * xh) + np.abs(dys) * xh_err).sum(0) + 1e-44)
    if db is not None:
        assert np.all(np.abs(_np(db) - dbr) <= down * U * np.abs(dys).sum(0) + 1e-44)


SIZES = [(1, 1), (1, 7), (3, 8), (2, 128), (65, 128), (1000, 96), (5, 129), (77, 1000), (33, 2048), (9, 5003),
         (700, 256), (3, 8192), (2, 8193), (70, 9000), (1, 40000)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,n", SIZES)
@pytest.mark.parametrize("rms,affine", [(False, True), (True, True), (False, False)])
def test_norm_and_its_gradients_match_fp64(rows, n, dtype, rms, affine):
    from pretraining_optimizer_b200 import layer_norm, layer_norm_backward
    x, dy, w, b = _data(rows, n, _dtype(dtype))
    if not affine:
        w = b = None
    y, mean, rstd = layer_norm(x, w, b, eps=1e-6, rms=rms)
    assert y.shape == x.shape and y.dtype == x.dtype and (mean is None) == rms and rstd.shape == (rows,)
    check_forward(x, w, b, 1e-6, rms, y, mean, rstd)
    dx, dw, db = layer_norm_backward(dy, x, w, mean, rstd, bias=affine)
    assert (dw is None) == (db is None) == (not affine)
    check_backward(dy, x, w, mean, rstd, dx, dw, db)


@pytest.mark.parametrize("n,extra,offset", [(128, 8, 0), (128, 3, 0), (128, 8, 1), (1001, 7, 2), (2048, 64, 8)])
def test_strided_and_unaligned_rows(n, extra, offset):
    """Rows of a wider buffer, at any offset: only the n columns of a row count."""
    t = _t()
    from pretraining_optimizer_b200 import layer_norm, layer_norm_backward
    x, dy, w, b = _data(37, n, t.bfloat16)
    wide = t.full((37, n + extra + offset), float("nan"), dtype=t.bfloat16, device="cuda:0")
    view = wide[:, offset:offset + n]
    view.copy_(x)
    target = t.full((37, n + extra + offset), 7.0, dtype=t.bfloat16, device="cuda:0")
    y, mean, rstd = layer_norm(view, w, b, out=target[:, offset:offset + n])
    check_forward(x, w, b, 1e-5, False, y, mean, rstd)
    assert bool((target[:, :offset] == 7).all()) and bool((target[:, offset + n:] == 7).all())
    wide_dy = t.full((37, n + extra), float("nan"), dtype=t.bfloat16, device="cuda:0")
    wide_dy[:, :n].copy_(dy)
    dx, dw, db = layer_norm_backward(wide_dy[:, :n], view, w, mean, rstd, bias=True)
    check_backward(dy, x, w, mean, rstd, dx, dw, db)


def test_leading_dimensions_and_in_place():
    t = _t()
    from pretraining_optimizer_b200 import layer_norm
    x, _, w, _ = _data(24, 128, t.float32)
    ref, mean, rstd = layer_norm(x, w)
    cube = x.clone().view(2, 3, 4, 128)
    y, m, r = layer_norm(cube, w, out=cube)
    assert y is cube and m.shape == (2, 3, 4)
    assert t.equal(cube.view(24, 128), ref) and t.equal(m.reshape(-1), mean) and t.equal(r.reshape(-1), rstd)


def test_heads_of_a_projection_as_rows():
    """The q norm: [tokens, heads, 128] rows inside a wider projection."""
    t = _t()
    from pretraining_optimizer_b200 import layer_norm, layer_norm_backward
    rng = np.random.default_rng(3)
    qkv = t.from_numpy(rng.standard_normal((50, 4096))).to("cuda:0", t.bfloat16)
    one = qkv[:, :128]
    w = t.ones(128, device="cuda:0")
    y, _, rstd = layer_norm(one, w, rms=True)
    check_forward(one.contiguous(), w, None, 1e-5, True, y, None, rstd)
    dx, dw, _ = layer_norm_backward(one, one, w, None, rstd)
    check_backward(one.contiguous(), one.contiguous(), w, None, rstd, dx, dw, None)


def test_gradients_match_differences():
    """A directional derivative of sum(y c) against central differences, in fp32 with fp64 sums:
    the difference's own error is u |loss| / h + h^2 f'''/6, with h = 2^-8 at unit scale."""
    t = _t()
    from pretraining_optimizer_b200 import layer_norm, layer_norm_backward
    g = t.Generator(device="cuda").manual_seed(1)
    x, c, dxn = (t.randn(16, 257, generator=g, device="cuda") for _ in range(3))
    w, b, dwn, dbn = (t.randn(257, generator=g, device="cuda") for _ in range(4))
    h = 2.0 ** -8

    def loss(k):
        y, _, _ = layer_norm(x + k * dxn, w + k * dwn, b + k * dbn)
        return float((y.double() * c.double()).sum())

    y, mean, rstd = layer_norm(x, w, b)
    dx, dw, db = layer_norm_backward(c, x, w, mean, rstd, bias=True)
    along = float((dx.double() * dxn).sum() + (dw.double() * dwn).sum() + (db.double() * dbn).sum())
    diff = (loss(h) - loss(-h)) / (2 * h)
    # rounding: every y is off by some 8 u |y|, 4112 of them with random signs over 2 h; third derivative of
    # x-hat along a unit direction is below 30 per element
    scale = float((y.abs() * c.abs()).double().square().sum().sqrt())
    bound = 8 * U * scale / h + h * h * 5 * float(c.abs().double().sum())
    assert abs(along - diff) <= bound, (along, diff, bound)


def test_rows_with_nan_or_infinity_leave_the_others_alone():
    t = _t()
    from pretraining_optimizer_b200 import layer_norm
    x, _, w, b = _data(9, 300, t.float32)
    clean, _, _ = layer_norm(x, w, b)
    x[2, 5], x[6, 299] = float("nan"), float("inf")
    y, _, rstd = layer_norm(x, w, b)
    assert bool(y[2].isnan().all()) and bool(y[6].isnan().any())
    keep = [0, 1, 3, 4, 5, 7, 8]
    assert t.equal(y[keep], clean[keep])


def test_constant_and_zero_rows():
    t = _t()
    from pretraining_optimizer_b200 import layer_norm
    x = t.zeros(2, 64, device="cuda:0")
    x[1] = 3.0
    y, mean, rstd = layer_norm(x, eps=1e-6)
    assert bool((y == 0).all()) and mean.tolist() == [0.0, 3.0]
    assert np.allclose(rstd.cpu().numpy(), 1e3, rtol=4 * U + 2 ** -23)


def test_no_rows():
    t = _t()
    from pretraining_optimizer_b200 import layer_norm, layer_norm_backward
    x = t.empty(0, 64, device="cuda:0")
    w = t.ones(64, device="cuda:0")
    y, mean, rstd = layer_norm(x, w)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dw, db = layer_norm_backward(x, x, w, mean, rstd, bias=True)
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())


def test_the_same_bits_every_time_on_any_stream():
    t = _t()
    from pretraining_optimizer_b200 import layer_norm, layer_norm_backward
    x, dy, w, b = _data(3001, 640, t.bfloat16)
    y, mean, rstd = layer_norm(x, w, b)
    first = layer_norm_backward(dy, x, w, mean, rstd, bias=True)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    for stream in (None, side, None, side):
        again = layer_norm_backward(dy, x, w, mean, rstd, bias=True, stream=stream)
        t.cuda.synchronize()
        assert all(t.equal(a, c) for a, c in zip(first, again))


def test_captured_in_a_graph():
    t = _t()
    from pretraining_optimizer_b200 import layer_norm, layer_norm_backward
    x, dy, w, b = _data(200, 512, t.bfloat16)
    x2, dy2, _, _ = _data(200, 512, t.bfloat16, seed=9)
    layer_norm(x, w, b)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        y, mean, rstd = layer_norm(x, w, b)
        grads = layer_norm_backward(dy, x, w, mean, rstd, bias=True)
    x.copy_(x2)
    dy.copy_(dy2)
    graph.replay()
    t.cuda.synchronize()
    want, m2, r2 = layer_norm(x2, w, b)
    want_grads = layer_norm_backward(dy2, x2, w, m2, r2, bias=True)
    assert t.equal(y, want) and all(t.equal(a, c) for a, c in zip(grads, want_grads))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [64, 65, 256, 257, 512, 513, 520, 1024, 1028, 2047, 2048, 2052, 4096, 4097, 4100, 8190])
def test_widths_around_the_kernels_borders(n, dtype):
    """Both sides of every change of kernel and of threads per row, with more rows than groups of threads."""
    from pretraining_optimizer_b200 import layer_norm, layer_norm_backward
    rows = 1400 if n <= 4096 else 700
    x, dy, w, b = _data(rows, n, _dtype(dtype), seed=n)
    y, mean, rstd = layer_norm(x, w, b, eps=1e-6)
    check_forward(x, w, b, 1e-6, False, y, mean, rstd)
    check_backward(dy, x, w, mean, rstd, *layer_norm_backward(dy, x, w, mean, rstd, bias=True))


@pytest.mark.parametrize("n", [100, 777, 3000])
def test_each_combination_of_gradients(n):
    t = _t()
    from pretraining_optimizer_b200 import layer_norm, layer_norm_backward
    x, dy, w, _ = _data(333, n, t.bfloat16)
    _, mean, rstd = layer_norm(x, w)
    dx, dw, db = layer_norm_backward(dy, x, w, mean, rstd, bias=True)
    alone, dw2, none = layer_norm_backward(dy, x, w, mean, rstd)
    assert none is None and t.equal(alone, dx) and t.equal(dw2, dw)
    plain, none, db2 = layer_norm_backward(dy, x, None, mean, rstd, bias=True)
    assert none is None and t.equal(db2, db)
    check_backward(dy, x, None, mean, rstd, plain, None, db2)
    rows_only = layer_norm_backward(dy, x, None, mean, rstd)
    assert rows_only[1:] == (None, None) and t.equal(rows_only[0], plain)


@pytest.mark.parametrize("n", [127, 1001, 5003, 9001])
def test_unaligned_rows_in_place(n):
    """Neighbouring rows share 16-byte pieces; writing a row leaves the others as they are."""
    t = _t()
    from pretraining_optimizer_b200 import layer_norm
    x, _, w, b = _data(900, n, t.bfloat16)
    ref, _, _ = layer_norm(x, w, b)
    got, _, _ = layer_norm(x, w, b, out=x)
    assert got is x and t.equal(x, ref)


def test_on_a_side_stream_after_its_own_work():
    """A call on a stream sees what that stream did before, and its results belong to it."""
    t = _t()
    from pretraining_optimizer_b200 import layer_norm, layer_norm_backward
    x, dy, w, b = _data(4000, 1024, t.bfloat16)
    want = layer_norm_backward(dy, x, w, *layer_norm(x, w, b)[1:], bias=True)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        late = t.zeros_like(x)
        for _ in range(20):
            late.mul_(2.0)
        late.copy_(x)
    y, mean, rstd = layer_norm(late, w, b, stream=side)
    got = layer_norm_backward(dy, late, w, mean, rstd, bias=True, stream=side)
    side.synchronize()
    assert all(t.equal(a, c) for a, c in zip(want, got))
