"""Block-scaled 8-bit quantising and products vs fp64 (B200 only).

Quantising is exact: values and scales have to be equal.  A product's tolerance
is in units of S = sum_k |a b| of each element.  An MMA adds 32 products to the
accumulator and truncates: it loses at most one step of fp32 (2^-23) of the sum
and, where it aligns the products to the largest, as much again, so 2^-22 S per
MMA.  There are four per 128 of k, counted over at most 32 such blocks for fp32
results, whose chunks are added in fp32 (2^-24 S each); a 16-bit result counts
all of k, and is rounded once (half a step)."""
import numpy as np
import pytest

from oracle import operators as O

pytestmark = pytest.mark.gpu


def _t():
    import torch
    return torch


def _dtype(name):
    t = _t()
    return {"fp32": t.float32, "bf16": t.bfloat16, "fp16": t.float16}[name]


def _data(rows, cols, seed=0, spread=2.0):
    rng = np.random.default_rng(seed)
    return rng.standard_normal((rows, cols)) * np.exp(spread * rng.standard_normal((rows, 1)))


def _np(x):
    return x.to(_t().float64).cpu().numpy() if x.is_floating_point() else x.cpu().numpy()


def check_quantized(x, q, s, block_rows):
    xs = _np(x)
    qr, sr = O.block_quantize(xs, block_rows)
    assert np.array_equal(s.cpu().numpy(), sr)
    assert q.shape == x.shape and (q.shape[0] < 2 or q.stride(0) % 16 == 0)
    assert np.array_equal(_np(q.float()), qr)


SIZES = [(1, 1), (1, 128), (3, 5), (128, 128), (129, 130), (77, 1000), (300, 136), (260, 2048), (1, 4097)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize_matches_the_definition(rows, cols, dtype):
    t = _t()
    from pretraining_optimizer_b200 import block_quantize, block_quantize_weight
    x = t.from_numpy(_data(rows, cols, rows)).to("cuda:0", _dtype(dtype))
    q, s, qt, st = block_quantize(x, columns=True)
    check_quantized(x, q, s, 1)
    check_quantized(x.t(), qt, st, 1)
    only = block_quantize(x)
    assert t.equal(only[0].view(t.uint8), q.view(t.uint8)) and t.equal(only[1], s)
    only = block_quantize(x, rows=False, columns=True)
    assert t.equal(only[0].view(t.uint8), qt.view(t.uint8)) and t.equal(only[1], st)
    q, s, qt, st = block_quantize_weight(x)
    check_quantized(x, q, s, 128)
    check_quantized(x.t(), qt, st, 128)


def test_quantize_borders():
    """Largest magnitudes on both sides of 448 2^k, ties, the smallest and largest scales, zeros."""
    t = _t()
    from pretraining_optimizer_b200 import block_quantize
    x = np.zeros((12, 128), dtype=np.float32)
    x[0, 3], x[1, 3], x[2, 3] = 448.0, np.nextafter(np.float32(448), np.float32(500)), 896.0
    x[3, 3], x[4, 3] = 2.0 ** -140, 3.4e38
    x[5, :4] = 448.0, 1.0625, 1.1875, -1.0625          # ties between neighbours
    x[6, :3] = 448.0, 2.0 ** -10, 3 * 2.0 ** -10        # ties among the smallest
    x[7] = -1e-3
    x[9] = np.linspace(-300, 300, 128)
    x[10, 0], x[11, 0] = 2.0 ** -127, -1.75 * 2.0 ** 20
    d = t.from_numpy(x).to("cuda:0")
    q, s = block_quantize(d)
    check_quantized(d, q, s, 1)
    assert s[8, 0] == 127 and s[3, 0] == 0 and s[4, 0] == 127 + 120


def test_quantize_rows_of_a_wider_buffer():
    t = _t()
    from pretraining_optimizer_b200 import block_quantize
    x = t.from_numpy(_data(150, 200)).to("cuda:0", t.bfloat16)
    for offset, width in ((0, 208), (8, 208), (3, 207)):
        wide = t.full((150, width + 8), float("nan"), dtype=t.bfloat16, device="cuda:0")
        wide[:, offset:offset + 200] = x
        q, s, qt, st = block_quantize(wide[:, offset:offset + 200], columns=True)
        check_quantized(x, q, s, 1)
        check_quantized(x.t(), qt, st, 1)


def test_quantize_leaves_the_padding_alone():
    t = _t()
    from pretraining_optimizer_b200 import muonh as B
    x = t.from_numpy(_data(5, 21)).to("cuda:0", t.float32)
    q = t.full((7, 48), 9, dtype=t.uint8, device="cuda:0")
    s = t.full((7, 3), 9, dtype=t.uint8, device="cuda:0")
    B._check(B.library().muonh_block_quantize(x.data_ptr(), 21, 5, 21, 0, 1, q[1].data_ptr(), 48, s[1].data_ptr(), 3,
                                              None, 0, None, 0, t.cuda.current_stream().cuda_stream))
    t.cuda.synchronize()
    check_quantized(x, q[1:6, :21].view(t.float8_e4m3fn), s[1:6, :1], 1)
    q[1:6, :21] = 9
    s[1:6, :1] = 9
    assert bool((q == 9).all()) and bool((s == 9).all())


def test_non_finite_groups_are_nan():
    t = _t()
    from pretraining_optimizer_b200 import block_matmul, block_quantize
    x = t.from_numpy(_data(4, 256, spread=0.0)).to("cuda:0", t.float32)
    clean = block_quantize(x)
    x[1, 130], x[2, 5] = float("nan"), float("-inf")
    q, s = block_quantize(x)
    assert s[1].tolist()[1] == 255 and s[2].tolist()[0] == 255
    assert bool(q[1, 128:].float().isnan().all()) and bool(q[2, :128].float().isnan().all())
    assert t.equal(q[0].view(t.uint8), clean[0][0].view(t.uint8)) and t.equal(q[1, :128].view(t.uint8), clean[0][1, :128].view(t.uint8))
    d = block_matmul(q, s, *clean, dtype=t.float32)
    assert bool(d[1].isnan().all()) and bool(d[2].isnan().all()) and bool(d[[0, 3]].isfinite().all())


def _operand(rng, rows, k, block_rows):
    """Small whole numbers in e4m3 and scales between 2^-3 and 2^3: products are exact in fp32."""
    t = _t()
    q = t.from_numpy(rng.integers(-2, 3, (rows, k)).astype(np.float32)).to("cuda:0")
    room = t.zeros(rows, -(-k // 16) * 16, dtype=t.float8_e4m3fn, device="cuda:0")[:, :k]
    room.copy_(q.to(t.float8_e4m3fn))
    s = t.from_numpy(rng.integers(124, 131, (-(-rows // block_rows), -(-k // 128))).astype(np.uint8)).to("cuda:0")
    return room, s


PRODUCTS = [(1, 1, 1), (1, 64, 128), (3, 7, 33), (128, 128, 128), (130, 70, 260), (77, 520, 1000), (128, 256, 512),
            (300, 257, 640), (64, 2048, 896), (2500, 1900, 400), (3000, 2700, 1160),
            (100, 200, 9000), (5, 3, 1024), (260, 70, 5000), (2300, 2310, 4300), (256, 256, 128), (1700, 1500, 136)]


@pytest.mark.parametrize("blocks", [(1, 1), (1, 128), (128, 1), (128, 128)])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_products_of_whole_numbers_are_exact(m, n, k, blocks):
    """Every scale in its place: nothing is rounded, so the fp32 result is the exact one."""
    t = _t()
    from pretraining_optimizer_b200 import block_matmul, operator_status
    rng = np.random.default_rng(m + n + k)
    a, sa = _operand(rng, m, k, blocks[0])
    b, sb = _operand(rng, n, k, blocks[1])
    ref = O.block_values(a.float().cpu().numpy(), sa.cpu().numpy()) @ O.block_values(b.float().cpu().numpy(), sb.cpu().numpy()).T
    d = block_matmul(a, sa, b, sb, dtype=t.float32)
    operator_status()
    assert np.array_equal(_np(d), ref)
    start = t.from_numpy(rng.integers(-9, 10, (m, n)).astype(np.float32)).to("cuda:0")
    total = start.clone()
    assert block_matmul(a, sa, b, sb, out=total, accumulate=True) is total
    assert np.array_equal(_np(total), ref + _np(start))


def check_product(a, b, d, k):
    t = _t()
    ref, size = a @ b.T, np.abs(a) @ np.abs(b).T
    blocks = -(-k // 128)
    if d.dtype == t.float32:
        tol = (4 * min(blocks, 32) * 2.0 ** -22 + -(-blocks // 32) * 2.0 ** -24) * size
    else:
        tol = 4 * blocks * 2.0 ** -22 * size
        f = t.finfo(d.dtype)
        tol = tol + f.eps / 2 * (np.abs(ref) + tol) + f.smallest_normal * f.eps / 2
    assert np.all(np.abs(_np(d) - ref) <= tol + 1e-44), np.max(np.abs(_np(d) - ref) / (tol + 1e-44))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("m,n,k", [(77, 520, 1000), (1, 300, 2048), (513, 129, 4100), (700, 1000, 200), (256, 128, 16384)])
def test_quantised_products_match_fp64(m, n, k, dtype):
    t = _t()
    from pretraining_optimizer_b200 import block_matmul, block_quantize, block_quantize_weight
    x = t.from_numpy(_data(m, k, 1, 1.0)).to("cuda:0", t.bfloat16)
    w = t.from_numpy(0.02 * _data(n, k, 2, 0.0)).to("cuda:0", t.float32)
    q, s = block_quantize(x)
    wq, ws, _, _ = block_quantize_weight(w)
    d = block_matmul(q, s, wq, ws, dtype=_dtype(dtype))
    check_product(O.block_values(q.float().cpu().numpy(), s.cpu().numpy()),
                  O.block_values(wq.float().cpu().numpy(), ws.cpu().numpy()), d, k)


def test_a_layer_forward_and_backward():
    """The three products of a linear layer from their quantised operands; the weight gradient is added to."""
    t = _t()
    from pretraining_optimizer_b200 import block_matmul, block_quantize, block_quantize_weight
    tokens, inputs, outputs = 333, 400, 260
    x = t.from_numpy(_data(tokens, inputs, 1, 1.0)).to("cuda:0", t.bfloat16)
    dy = t.from_numpy(1e-3 * _data(tokens, outputs, 2, 1.0)).to("cuda:0", t.bfloat16)
    w = t.from_numpy(0.02 * _data(outputs, inputs, 3, 0.0)).to("cuda:0", t.float32)
    value = lambda q, s: O.block_values(q.float().cpu().numpy(), s.cpu().numpy())  # noqa: E731
    xq, xs, xt, xts = block_quantize(x, columns=True)
    wq, ws, wt, wts = block_quantize_weight(w)
    g, gs, gt, gts = block_quantize(dy, columns=True)
    check_product(value(xq, xs), value(wq, ws), block_matmul(xq, xs, wq, ws), inputs)
    check_product(value(g, gs), value(wt, wts), block_matmul(g, gs, wt, wts), outputs)
    grad = t.zeros(outputs, inputs, device="cuda:0")
    block_matmul(gt, gts, xt, xts, out=grad, accumulate=True)
    check_product(value(gt, gts), value(xt, xts), grad, tokens)
    # the quantised layer is near the layer itself: each operand is off by at most 2^-4 relative (e4m3 with
    # values below 2^-6 448 of the group's largest rounded to a step of 2^-9 / 448 of it)
    exact = _np(dy).T @ _np(x)
    assert np.linalg.norm(_np(grad) - exact) <= (2 * 2.0 ** -4 + 2.0 ** -8) * np.linalg.norm(np.abs(_np(dy)).T @ np.abs(_np(x)))


def test_products_into_strided_results():
    t = _t()
    from pretraining_optimizer_b200 import block_matmul
    rng = np.random.default_rng(3)
    a, sa = _operand(rng, 140, 300, 1)
    b, sb = _operand(rng, 90, 300, 1)
    ref = block_matmul(a, sa, b, sb, dtype=t.float32)
    for dtype, offset in ((t.float32, 0), (t.float32, 3), (t.bfloat16, 1), (t.float16, 16)):
        wide = t.full((142, 120), 5.0, dtype=dtype, device="cuda:0")
        view = wide[1:-1, offset:offset + 90]
        block_matmul(a, sa, b, sb, out=view)
        assert t.equal(view, ref.to(dtype))
        view.fill_(5.0)
        assert bool((wide == 5.0).all())


def test_products_of_operands_inside_wider_buffers():
    """Row strides above k, and scales that no 4-byte load can address."""
    t = _t()
    from pretraining_optimizer_b200 import block_matmul
    rng = np.random.default_rng(4)
    a, sa = _operand(rng, 200, 640, 1)
    b, sb = _operand(rng, 150, 640, 1)
    ref = block_matmul(a, sa, b, sb, dtype=t.float32)
    wide = t.full((200, 1280), float("nan"), device="cuda:0").to(t.float8_e4m3fn)
    wide[:, 640:].copy_(a)
    scales = t.full((200, 12), 255, dtype=t.uint8, device="cuda:0")
    for at in (0, 1, 4, 7):
        scales.fill_(255)
        scales[:, at:at + 5] = sa
        got = block_matmul(wide[:, 640:], scales[:, at:at + 5], b, sb, dtype=t.float32)
        assert t.equal(got, ref)


def test_empty_products():
    t = _t()
    from pretraining_optimizer_b200 import block_matmul, block_quantize
    q0, s0 = block_quantize(t.empty(0, 64, device="cuda:0"))
    q, s = block_quantize(t.ones(3, 64, device="cuda:0"))
    assert block_matmul(q0, s0, q, s).shape == (0, 3) and block_matmul(q, s, q0, s0).shape == (3, 0)
    e, es = block_quantize(t.empty(3, 0, device="cuda:0"))
    out = t.full((3, 3), 7.0, device="cuda:0")
    block_matmul(e, es, e, es, out=out, accumulate=True)
    assert bool((out == 7).all())
    block_matmul(e, es, e, es, out=out)
    assert bool((out == 0).all())


def test_the_same_bits_on_any_stream_and_in_a_graph():
    t = _t()
    from pretraining_optimizer_b200 import block_matmul, block_quantize, operator_status
    x = t.from_numpy(_data(520, 1200, 1)).to("cuda:0", t.bfloat16)
    y = t.from_numpy(_data(390, 1200, 2)).to("cuda:0", t.bfloat16)
    b, sb = block_quantize(y)

    def layer(stream=None):
        q, s = block_quantize(x, stream=stream)
        return block_matmul(q, s, b, sb, dtype=t.float32, stream=stream)

    first = layer()
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    for _ in range(3):
        one, two = layer(), layer(side)
        t.cuda.synchronize()
        assert t.equal(one, first) and t.equal(two, first)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        got = layer()
    x.copy_(t.from_numpy(_data(520, 1200, 5)).to(x))
    graph.replay()
    t.cuda.synchronize()
    assert t.equal(got, layer())
    operator_status()


def test_an_operand_with_itself_and_results_that_alternate():
    """The same operand on both sides, and calls that follow each other without a wait."""
    t = _t()
    from pretraining_optimizer_b200 import block_matmul
    rng = np.random.default_rng(8)
    a, sa = _operand(rng, 300, 700, 1)
    va = O.block_values(a.float().cpu().numpy(), sa.cpu().numpy())
    b, sb = _operand(rng, 2100, 700, 128)
    vb = O.block_values(b.float().cpu().numpy(), sb.cpu().numpy())
    results = []
    for _ in range(5):
        results.append((block_matmul(a, sa, a, sa, dtype=t.float32), block_matmul(b, sb, b, sb, dtype=t.float32)))
    for small, large in results:
        assert np.array_equal(_np(small), va @ va.T) and np.array_equal(_np(large), vb @ vb.T)


def test_refusals_of_the_binding():
    t = _t()
    from pretraining_optimizer_b200 import MuonHError, block_matmul, block_quantize
    q, s = block_quantize(t.ones(40, 200, device="cuda:0"))
    r, rs = block_quantize(t.ones(30, 200, device="cuda:0"))
    with pytest.raises(ValueError):
        block_matmul(q, s[:, :1], r, rs)                      # too few scales
    with pytest.raises(ValueError):
        block_matmul(q, s[:7], r, rs)
    with pytest.raises(ValueError):
        block_matmul(q[:, :128], s[:, :1], r, rs)             # different k
    with pytest.raises(MuonHError):
        block_matmul(q.contiguous(), s, r, rs)                # rows of 200 bytes: not 16-byte aligned
    with pytest.raises(TypeError):
        block_matmul(q, s, r, rs, dtype=t.float64)
    with pytest.raises(ValueError):
        block_matmul(q, s, r, rs, accumulate=True)            # nothing to add to
    with pytest.raises(MuonHError):
        block_matmul(q, s, r, rs, out=t.zeros(40, 30, dtype=t.bfloat16, device="cuda:0"), accumulate=True)
    with pytest.raises(ValueError):
        block_matmul(q, s, r, rs, out=t.zeros(30, 40, device="cuda:0"))
    with pytest.raises(ValueError):
        block_quantize(t.ones(4, 8, 8, device="cuda:0"))
    with pytest.raises(ValueError):
        block_quantize(t.ones(8, 8, device="cuda:0").t()[:, ::2])
