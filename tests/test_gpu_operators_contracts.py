"""What the operators' documentation promises at the edges: non-finite rows and matrices, results' layouts, and
in-place writes that autograd has to see (B200 only)."""
import pytest

pytestmark = pytest.mark.gpu


def _randn(seed, *shape):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("steps", [0, 1, 2, 5, 6])
def test_a_matrix_with_infinity_is_nan_throughout_at_every_step_count(steps, dtype):
    import torch
    from pretraining_optimizer_b200 import orthogonalize
    for shape in ((4, 40, 96), (4, 96, 40), (4, 128, 700)):
        x = _randn(1, *shape).to({"bf16": torch.bfloat16, "fp16": torch.float16}[dtype])
        clean = orthogonalize(x, ns_steps=steps)
        x[1, 3, 5], x[2, 39, 39], x[3, 0, 0] = float("inf"), float("-inf"), float("nan")
        got = orthogonalize(x, ns_steps=steps)
        assert torch.equal(got[0], clean[0])
        assert bool(got[1:].isnan().all())
        # finite, with a norm beyond fp32's square: NaN in pairs, and within fp64
        if dtype == "bf16":
            huge = orthogonalize(x[:1] * 2.0 ** 66, ns_steps=steps)
            assert bool(huge.isnan().all()) if steps <= 5 else bool(huge.isfinite().all())


@pytest.mark.parametrize("n", [100, 300, 2048, 9000])
@pytest.mark.parametrize("rms", [False, True])
def test_rows_with_nan_or_infinity(rms, n):
    """NaN: the row is NaN.  Inf: NaN for the layer norm; for the RMS norm rstd is 0, so the infinite elements are NaN
    and the finite ones the bias."""
    import torch
    from pretraining_optimizer_b200 import layer_norm
    x, w, b = _randn(2, 9, n), _randn(3, n), _randn(4, n)
    clean, _, clean_rstd = layer_norm(x, w, b, rms=rms)
    x[2, 5], x[6, n - 1], x[7, 0] = float("nan"), float("inf"), float("-inf")
    y, _, rstd = layer_norm(x, w, b, rms=rms)
    assert bool(y[2].isnan().all()) and bool(rstd[2].isnan())
    for row, at in ((6, n - 1), (7, 0)):
        if rms:
            finite = torch.arange(n, device="cuda") != at
            assert float(rstd[row]) == 0 and bool(y[row, at].isnan()) and torch.equal(y[row, finite], b[finite])
        else:
            assert bool(y[row].isnan().all()) and bool(rstd[row].isnan())
    keep = [0, 1, 3, 4, 5, 8]
    assert torch.equal(y[keep], clean[keep]) and torch.equal(rstd[keep], clean_rstd[keep])


def test_matrices_that_overlap_in_the_input():
    """A window that slides over one buffer: any batch stride is allowed on the way in."""
    import torch
    from pretraining_optimizer_b200 import orthogonalize
    buffer = _randn(5, 4000).bfloat16()
    for shape, stride in (((4, 1, 8), (1, 8, 1)), ((4, 3, 8), (1, 8, 1)), ((5, 16, 40), (3, 40, 1)), ((3, 4, 8), (0, 8, 1)),
                          ((6, 16, 40), (40, 40, 1))):
        x = buffer.as_strided(shape, stride)
        got = orthogonalize(x)
        assert got.shape == x.shape and torch.equal(got, orthogonalize(x.contiguous()))
        # the result's matrices are apart: clearing one leaves the others
        want = got.clone()
        want[0] = 0
        got[0] = 0
        assert torch.equal(got, want)


def test_results_whose_matrices_overlap_are_refused():
    import torch
    from pretraining_optimizer_b200 import orthogonalize
    buffer = torch.zeros(20000, device="cuda", dtype=torch.bfloat16)
    for shape, stride in (((3, 4, 8), (8, 8, 1)), ((3, 4, 8), (24, 8, 1)), ((3, 4, 8), (12, 16, 1)), ((9, 4, 8), (8, 64, 1)),
                          ((2, 3, 5), (20, 10, 1)), ((2, 4, 8), (4, 8, 1)), ((2, 4, 8), (0, 8, 1))):
        x = _randn(6, *shape).bfloat16()
        with pytest.raises(ValueError, match="overlap"):
            orthogonalize(x, out=buffer.as_strided(shape, stride))
    assert not bool(buffer.any())
    # one behind the other, side by side, and row by row in turn
    for shape, stride in (((3, 4, 8), (32, 8, 1)), ((3, 4, 8), (40, 8, 1)), ((8, 4, 8), (8, 64, 1)), ((2, 3, 5), (15, 10, 1)),
                          ((2, 3, 5), (5, 10, 1)), ((3, 1, 8), (8, 8, 1)), ((1, 4, 8), (0, 8, 1))):
        x = _randn(7, *shape).bfloat16()
        out = buffer.as_strided(shape, stride)
        assert torch.equal(orthogonalize(x, out=out), orthogonalize(x))


def test_writes_to_out_are_seen_by_autograd():
    """A tensor that a graph saved and an operator then overwrites may not go into its gradient unnoticed."""
    import torch
    import pretraining_optimizer_b200 as P
    q, s = P.block_quantize(_randn(8, 32, 128))
    calls = (lambda t: P.layer_norm(t, out=t), lambda t: P.block_matmul(q, s, q, s, out=t),
             lambda t: P.orthogonalize(t.bfloat16(), out=t))
    for call, dtype in zip(calls, (torch.float32, torch.float32, torch.bfloat16)):
        saved = _randn(9, 32, 32).to(dtype)
        w = torch.ones(32, 32, device="cuda", dtype=dtype, requires_grad=True)
        loss = (w * saved).sum()
        call(saved)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    with torch.inference_mode():
        t = _randn(10, 32, 32)
        P.layer_norm(t, out=t)


@pytest.mark.parametrize("shape", [(600, 64, 520), (610, 700, 33), (592, 128, 513), (591, 16, 1024), (600, 5, 4100)])
def test_stacks_whose_ctas_start_late(shape):
    """Four matrices per SM and more (and one fewer), with long sides on both sides of the late start's limit."""
    import torch
    from pretraining_optimizer_b200 import operator_status, orthogonalize
    from test_gpu_orthogonalize import check
    x = (1e-3 * _randn(11, *shape)).bfloat16()
    for steps in (0, 5):
        got = orthogonalize(x, ns_steps=steps)
        assert torch.equal(got, orthogonalize(x, ns_steps=steps))
        some = [0, 1, 147, 148, 149, shape[0] - 1]
        check(x[some], got[some], steps)
    operator_status()
