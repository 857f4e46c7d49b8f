"""orthogonalize where the factors grow far beyond one: many steps, other
coefficients, and matrices of low rank, whose empty directions grow by |a| in
each step while the result does not (B200 only).

Tolerance.  Up to a growth of 512 (five steps of the default coefficients are
485) the r x r iteration is kept in pairs; what is promised there is 1e-2 of
||out||, the step's own bound, beside the rounding of the result (half a step).
Most matrices here are held to less: 3e-3 for bf16 and 2e-3 for fp16, which the
same arithmetic with single fp16 operands fails.  Beyond it everything is fp64: an error of at most r 2^-52 of an operand
(products of at most 128 terms, and the long side's sum, whose terms' signs
vary) is amplified by the growth at most, and the result is rounded to fp32
(2^-24) on its way to 16 bits."""
import numpy as np
import pytest

from oracle import operators as O

pytestmark = pytest.mark.gpu

PAIRS = {"bf16": 3e-3, "fp16": 2e-3}
CUBIC = (1.5, -0.5, 0.0)


def _t():
    import torch
    return torch


def _dtype(name):
    t = _t()
    return {"bf16": t.bfloat16, "fp16": t.float16}[name]


def growth(steps, coeffs):
    """The largest |product of the factors| on the singular values that a matrix of norm one can have."""
    a, b, c = coeffs
    s, q = np.linspace(0, 1, 4001), np.ones(4001)
    for _ in range(steps):
        f = a + b * s ** 2 + c * s ** 4
        q, s = q * f, s * f
    return np.abs(q).max()


def matrices(kind, batch, r, c, seed=1):
    """exactK: whole numbers of rank K; K+e: rank K with noise e beside it; noise."""
    rng = np.random.default_rng(seed)
    if kind.startswith("exact"):
        k = int(kind[5:])
        return 2.0 ** -8 * (rng.integers(-3, 4, (batch, r, k)) @ rng.integers(-3, 4, (batch, k, c)))
    if "+" in kind:
        k, e = kind.split("+")
        low = rng.standard_normal((batch, r, int(k))) @ rng.standard_normal((batch, int(k), c))
        return 1e-3 * (low + float(e) * rng.standard_normal((batch, r, c)))
    return 1e-3 * rng.standard_normal((batch, r, c))


def check(x, got, steps, coeffs=O.QUINTIC, eps=1e-7, pairs_bound=None):
    t = _t()
    assert got.shape == x.shape and got.dtype == x.dtype
    xs, gs = x.double().cpu().numpy(), got.double().cpu().numpy()
    # the call takes its coefficients in fp32
    coeffs, eps = [float(np.float32(v)) for v in coeffs], float(np.float32(eps))
    ref = O.orthogonalize(xs, steps, coeffs, eps)
    g = growth(steps, coeffs)
    name = "bf16" if x.dtype == t.bfloat16 else "fp16"
    pairs = steps == 0 or (g <= 512 and abs(coeffs[0]) >= 1)
    half = t.finfo(x.dtype).eps / 2
    for i in range(xs.shape[0]):
        size = np.linalg.norm(ref[i])
        tol = (pairs_bound or PAIRS[name]) * size if pairs else 2.0 ** -24 * size + g * min(x.shape[-2:]) * 2.0 ** -52 * max(size, 1.0)
        tol += half * (size + tol)
        tol += (2.0 ** -25 if x.dtype == t.float16 else 0.0) * np.sqrt(ref[i].size) + 1e-30
        off = np.linalg.norm(gs[i] - ref[i])
        assert off <= tol, (i, off / size, tol / size)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("kind", ["exact1", "exact4", "8+1e-3", "1+1e-2", "noise"])
@pytest.mark.parametrize("steps", [1, 4, 5, 6, 8, 10, 16])
def test_steps_on_matrices_of_low_rank(steps, kind, dtype):
    t = _t()
    from pretraining_optimizer_b200 import operator_status, orthogonalize
    for shape in ((3, 128, 512), (2, 64, 64), (2, 300, 48), (4, 5, 5)):
        x = t.from_numpy(matrices(kind, *shape)).to("cuda:0", _dtype(dtype))
        check(x, orthogonalize(x, ns_steps=steps), steps)
    operator_status()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("kind", ["plain", "spiked", "rank"])
@pytest.mark.parametrize("shape", [(3, 128, 512), (2, 64, 64), (2, 128, 128), (2, 700, 128), (3, 48, 300), (1, 128, 8192)])
def test_five_steps_are_within_the_documented_bound(shape, kind, dtype):
    """Ill-conditioned updates, for which bounds from the spectrum alone are several times the result's norm."""
    t = _t()
    from pretraining_optimizer_b200 import orthogonalize
    from test_gpu_orthogonalize import _spectrum
    x = t.from_numpy(_spectrum(np.random.default_rng(4), *shape, kind)).to("cuda:0", _dtype(dtype))
    check(x, orthogonalize(x), 5)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("kind", ["exact1", "1+3e-4", "1+3e-3", "1+1e-2", "2+1e-2"])
@pytest.mark.parametrize("shape", [(32, 2, 8192), (32, 3, 1024), (16, 8192, 5), (16, 16, 9000), (8, 128, 1024), (600, 2, 2048)])
def test_the_promise_in_pairs_where_sums_are_long(shape, kind, dtype):
    """Directions of a hundredth and less of the largest next to long sums: what the tensor cores truncate while
    they add up X X^T and the r x r products is amplified by the square of the growth."""
    t = _t()
    from pretraining_optimizer_b200 import orthogonalize
    for coeffs, steps in ((O.QUINTIC, 5), ((2.0, -1.5, 0.5), 9)):
        x = t.from_numpy(matrices(kind, *shape, seed=10)).to("cuda:0", _dtype(dtype))
        x = x[x.abs().amax((1, 2)) > 0]
        check(x, orthogonalize(x, ns_steps=steps, ns_coeffs=coeffs), steps, coeffs, pairs_bound=1e-2)


@pytest.mark.parametrize("coeffs,steps", [(CUBIC, 15), (CUBIC, 16), ((2.0, -1.5, 0.5), 9), ((2.0, -1.5, 0.5), 10),
                                          ((20.0, -40.0, 21.0), 3), ((0.5, 0.25, 0.0), 6), ((0.0, 1.0, 0.0), 2),
                                          ((0.0, 0.0, 1.0), 1), ((-3.0, 3.0, -1.0), 4)])
def test_coefficients_that_grow_or_shrink(coeffs, steps):
    """Growth on both sides of the limit, factors that overflow 16 bits, and factors below one."""
    t = _t()
    from pretraining_optimizer_b200 import orthogonalize
    for kind in ("noise", "4+1e-2"):
        x = t.from_numpy(matrices(kind, 2, 48, 300)).to("cuda:0", t.bfloat16)
        check(x, orthogonalize(x, ns_steps=steps, ns_coeffs=coeffs), steps, coeffs)


def test_long_runs_of_every_layout():
    """Strided, unaligned, repeated and in place: the bits of the compact stack."""
    t = _t()
    from pretraining_optimizer_b200 import orthogonalize
    for shape in ((3, 24, 331), (3, 331, 24)):
        x = t.from_numpy(matrices("4+1e-2", *shape)).to("cuda:0", t.bfloat16)
        want = orthogonalize(x, ns_steps=8)
        check(x, want, 8)
        for offset, extra in ((1, 0), (0, 3), (3, 8)):
            wide = t.full((*shape[:2], shape[2] + offset + extra), float("nan"), dtype=t.bfloat16, device="cuda:0")
            view = wide[:, :, offset:offset + shape[2]]
            view.copy_(x)
            target = t.full_like(wide, 5.0)
            out = orthogonalize(view, ns_steps=8, out=target[:, :, offset:offset + shape[2]])
            assert t.equal(out, want)
            out.fill_(5.0)
            assert bool((target == 5.0).all())
            orthogonalize(view, ns_steps=8, out=view)
            assert t.equal(view, want)
        assert t.equal(orthogonalize(x[1], ns_steps=8), want[1])
        assert t.equal(orthogonalize(x[:1].expand(shape), ns_steps=8)[2], want[0])


def test_long_runs_of_large_and_small_stacks():
    """Stacks that the scratch holds in several parts, single rows and columns, and long sides."""
    t = _t()
    from pretraining_optimizer_b200 import orthogonalize
    for shape in ((230, 128, 136), (1, 128, 8192), (1, 41000, 16), (70000, 1, 3), (5, 7, 1), (1, 1, 1), (2, 127, 129)):
        x = t.from_numpy(matrices("noise", *shape)).to("cuda:0", t.float16)
        got = orthogonalize(x, ns_steps=7)
        some = [0, shape[0] // 2, shape[0] - 1]
        check(x[some], got[some], 7)
        if shape[0] == 230:
            check(x, got, 7)


def test_long_runs_of_zero_tiny_and_non_finite_matrices():
    t = _t()
    from pretraining_optimizer_b200 import orthogonalize
    x = t.from_numpy(matrices("noise", 6, 40, 96)).to("cuda:0", t.bfloat16)
    clean = orthogonalize(x, ns_steps=8)
    x[0] = 0
    x[1, 3, 5] = float("nan")
    x[2, 39, 95] = float("inf")
    x[3] *= 2.0 ** -60
    x[5] *= 2.0 ** 100
    got = orthogonalize(x, ns_steps=8)
    assert bool((got[0] == 0).all())
    assert bool(got[1].isnan().all()) and bool(got[2].isnan().all())
    assert t.equal(got[4], clean[4])
    check(x[3:4], got[3:4], 8)
    check(x[5:6], got[5:6], 8)
    assert bool((orthogonalize(x[:1], ns_steps=8, eps=0.0) == 0).all())


@pytest.mark.parametrize("cols", [264, 203])
def test_long_runs_of_matrices_far_apart(cols):
    """Matrices more than 2^31 elements apart: the bits of the compact stack, in place too."""
    t = _t()
    from pretraining_optimizer_b200 import orthogonalize
    x = t.from_numpy(matrices("4+1e-2", 3, 32, cols)).to("cuda:0", t.bfloat16)
    want = orthogonalize(x, ns_steps=8)
    far = 2 ** 31 + 64
    view = t.empty(2 * far + 32 * cols, dtype=t.bfloat16, device="cuda:0").as_strided(x.shape, (far, cols, 1))
    view.copy_(x)
    assert t.equal(orthogonalize(view, ns_steps=8).contiguous(), want)
    orthogonalize(view, ns_steps=8, out=view)
    assert t.equal(view.contiguous(), want)


def test_long_runs_on_a_side_stream_and_in_a_graph():
    t = _t()
    from pretraining_optimizer_b200 import orthogonalize
    x = t.from_numpy(matrices("4+1e-2", 20, 64, 200)).to("cuda:0", t.bfloat16)
    want = orthogonalize(x, ns_steps=8)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    for _ in range(3):
        a, b = orthogonalize(x, ns_steps=8), orthogonalize(x, ns_steps=8, stream=side)
        t.cuda.synchronize()
        assert t.equal(a, want) and t.equal(b, want)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        got = orthogonalize(x, ns_steps=8)
    x2 = t.from_numpy(matrices("4+1e-2", 20, 64, 200, seed=2)).to("cuda:0", t.bfloat16)
    x.copy_(x2)
    graph.replay()
    t.cuda.synchronize()
    assert t.equal(got, orthogonalize(x2, ns_steps=8))
