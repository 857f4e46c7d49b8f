"""Orthogonalising stacks of small matrices vs fp64 (B200 only).

Tolerance, per matrix, in the Frobenius norm.  O = Q(A) Y with A = Y Y^T and Q
the product of the steps' p(A_k).  An error E of A moves O, in A's eigenbasis,
by L_ij E_ij sigma_j, where L_ij = (Q(l_i) - Q(l_j)) / (l_i - l_j) (Q'(l_i) on
the diagonal).  A's entries carry the truncation of at most 128 accumulations
(2048 columns in steps of 16) of half a step of fp32 each on average, and of
the pairs' 22 bits: below d = 2^-17 of A's largest entry.  The later iterates'
errors are of the same kind and are amplified less; there are three products
per step, and counting each like the first gives (3 steps) d.  Q itself enters
the last product as a pair of X's type (2^-16 of an entry for bf16), and the
result is rounded once (half a step)."""
import numpy as np
import pytest

from oracle import operators as O

pytestmark = pytest.mark.gpu


def _t():
    import torch
    return torch


def _dtype(name):
    t = _t()
    return {"bf16": t.bfloat16, "fp16": t.float16}[name]


def _tolerance(x, steps, coeffs, eps, half_step, ref):
    """Frobenius tolerance for one matrix x (fp64) with the exact result ref."""
    if x.shape[0] > x.shape[1]:
        x = x.T
    y = x / (np.linalg.norm(x) + eps)
    gram = y @ y.T
    lam = np.clip(np.linalg.eigvalsh(gram), 0.0, None)

    def chain(l):
        """Q and its derivative at the eigenvalues l."""
        a, b, c = coeffs
        q, dq, dl = np.ones_like(l), np.zeros_like(l), np.ones_like(l)
        for _ in range(steps):
            p, dp = a + b * l + c * l * l, (b + 2 * c * l) * dl
            q, dq = q * p, dq * p + q * dp
            l, dl = l * p * p, dl * p * p + 2 * l * p * dp
        return q, dq

    q, dq = chain(lam)
    gap = lam[:, None] - lam[None, :]
    close = np.abs(gap) <= 1e-9 + 1e-6 * np.maximum(lam[:, None], lam[None, :])
    slope = np.where(close, np.maximum(np.abs(dq)[:, None], np.abs(dq)[None, :]),
                     np.abs(q[:, None] - q[None, :]) / np.where(close, 1.0, np.abs(gap)))
    d = 3 * max(steps, 1) * 2.0 ** -17 * np.abs(gram).max()
    moved = d * np.sqrt((slope ** 2 * lam[None, :]).sum())
    pair = 2.0 ** -16 * np.linalg.norm(q) * np.sqrt(lam.max())
    return half_step * np.linalg.norm(ref) + moved + pair


def _spectrum(rng, batch, r, c, kind):
    x = rng.standard_normal((batch, r, c))
    if kind == "spiked":      # noise over a few strong directions, as momentum looks
        k = max(1, min(4, r))
        x = x + rng.standard_normal((batch, r, k)) @ rng.standard_normal((batch, k, c))
    elif kind == "rank":      # nearly low rank
        k = max(1, min(8, r // 2))
        x = 1e-2 * x + rng.standard_normal((batch, r, k)) @ rng.standard_normal((batch, k, c))
    return 1e-3 * x


def check(x, got, steps=5, coeffs=O.QUINTIC, eps=1e-7):
    t = _t()
    assert got.shape == x.shape and got.dtype == x.dtype
    xs = x.double().cpu().numpy().reshape((-1,) + tuple(x.shape[-2:]))
    gs = got.double().cpu().numpy().reshape(xs.shape)
    ref = O.orthogonalize(xs, steps, coeffs, eps)
    half = t.finfo(x.dtype).eps / 2
    for i in range(xs.shape[0]):
        tol = _tolerance(xs[i], steps, coeffs, eps, half, ref[i]) + 1e-30
        # fp16 results below 2^-14 have a fixed spacing of 2^-24
        tol += (2.0 ** -25 if x.dtype == t.float16 else 0.0) * np.sqrt(ref[i].size)
        off = np.linalg.norm(gs[i] - ref[i])
        assert off <= tol, (i, off, tol, np.linalg.norm(ref[i]))


SHAPES = [(1, 1, 1), (3, 1, 7), (2, 5, 5), (4, 33, 200), (2, 128, 128), (3, 96, 1000), (2, 64, 2048), (1, 128, 8192),
          (160, 16, 256), (2, 200, 33), (3, 1000, 57), (1, 4096, 128), (2, 127, 129), (5, 129, 127), (2, 40, 201)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_matches_fp64(shape, dtype):
    t = _t()
    from pretraining_optimizer_b200 import operator_status, orthogonalize
    rng = np.random.default_rng(sum(shape))
    x = t.from_numpy(_spectrum(rng, *shape, "spiked")).to("cuda:0", _dtype(dtype))
    check(x, orthogonalize(x))
    operator_status()


@pytest.mark.parametrize("kind", ["plain", "rank"])
@pytest.mark.parametrize("shape", [(3, 128, 512), (2, 64, 64), (2, 700, 128)])
def test_other_spectra(kind, shape):
    t = _t()
    from pretraining_optimizer_b200 import orthogonalize
    x = t.from_numpy(_spectrum(np.random.default_rng(4), *shape, kind)).to("cuda:0", t.bfloat16)
    check(x, orthogonalize(x))


@pytest.mark.parametrize("steps", [0, 1, 2, 3, 8])
def test_step_counts(steps):
    t = _t()
    from pretraining_optimizer_b200 import orthogonalize
    x = t.from_numpy(_spectrum(np.random.default_rng(5), 2, 48, 300, "plain")).to("cuda:0", t.float16)
    check(x, orthogonalize(x, ns_steps=steps), steps)


def test_other_coefficients_and_eps():
    t = _t()
    from pretraining_optimizer_b200 import orthogonalize
    x = t.from_numpy(_spectrum(np.random.default_rng(6), 2, 48, 300, "plain")).to("cuda:0", t.bfloat16)
    coeffs = (1.875, -1.25, 0.375)
    check(x, orthogonalize(x, ns_steps=4, ns_coeffs=coeffs), 4, coeffs)
    check(x, orthogonalize(x, eps=0.5), eps=0.5)


@pytest.mark.parametrize("tall", [False, True])
def test_heads_inside_one_matrix(tall):
    """Heads as row blocks (queries) or column blocks (the output projection) of one weight's update;
    results land in the same places and nowhere else."""
    t = _t()
    from pretraining_optimizer_b200 import orthogonalize
    x = t.from_numpy(_spectrum(np.random.default_rng(7), 1, 1, 6 * 96 * 520, "plain")).to("cuda:0", t.bfloat16)
    whole = x.view(520, 576) if tall else x.view(576, 520)
    heads = whole.unflatten(1, (6, 96)).transpose(0, 1) if tall else whole.unflatten(0, (6, 96))
    copy = heads.contiguous()
    got = orthogonalize(heads)
    check(copy, got)
    target = t.full((whole.shape[0] + 2, whole.shape[1] + 16), 5.0, dtype=t.bfloat16, device="cuda:0")
    inner = target[1:-1, 8:-8]
    out = inner.unflatten(1, (6, 96)).transpose(0, 1) if tall else inner.unflatten(0, (6, 96))
    orthogonalize(heads, out=out)
    assert t.equal(out, got)
    target[1:-1, 8:-8] = 5.0
    assert bool((target == 5.0).all())


@pytest.mark.parametrize("offset,extra", [(1, 0), (0, 3), (3, 8)])
def test_unaligned_rows(offset, extra):
    """Rows that no 16-byte access can address, on the way in and out."""
    t = _t()
    from pretraining_optimizer_b200 import orthogonalize
    x = t.from_numpy(_spectrum(np.random.default_rng(8), 3, 24, 331, "plain")).to("cuda:0", t.bfloat16)
    ref = orthogonalize(x)
    check(x, ref)
    wide = t.full((3, 24, 331 + offset + extra), float("nan"), dtype=t.bfloat16, device="cuda:0")
    wide[:, :, offset:offset + 331] = x
    target = t.full_like(wide, 5.0)
    out = orthogonalize(wide[:, :, offset:offset + 331], out=target[:, :, offset:offset + 331])
    assert t.equal(out, ref)
    out.fill_(5.0)
    assert bool((target == 5.0).all())


def test_in_place_and_single_matrix():
    t = _t()
    from pretraining_optimizer_b200 import orthogonalize
    x = t.from_numpy(_spectrum(np.random.default_rng(9), 5, 128, 1024, "plain")).to("cuda:0", t.bfloat16)
    ref = orthogonalize(x)
    one = orthogonalize(x[2])
    # a single matrix may be shared by more CTAs, whose Gram shares add up in another order
    check(x[2], one)
    y = x.clone()
    assert orthogonalize(y, out=y) is y and t.equal(y, ref)


def test_repeated_matrix():
    """A batch stride of zero: the same matrix at every index."""
    t = _t()
    from pretraining_optimizer_b200 import orthogonalize
    x = t.from_numpy(_spectrum(np.random.default_rng(10), 1, 32, 64, "plain")).to("cuda:0", t.bfloat16)
    got = orthogonalize(x.expand(3, 32, 64))
    assert all(t.equal(got[i], got[0]) for i in range(3))
    check(x, got[:1])


def test_zero_tiny_and_non_finite_matrices():
    """Zeros give zeros, NaN and Inf give NaN in their own matrix only, and a norm far below eps is divided by eps."""
    t = _t()
    from pretraining_optimizer_b200 import orthogonalize
    x = t.from_numpy(_spectrum(np.random.default_rng(11), 5, 40, 96, "plain")).to("cuda:0", t.bfloat16)
    clean = orthogonalize(x)
    x[0] = 0
    x[1, 3, 5] = float("nan")
    x[2, 39, 95] = float("inf")
    x[3] *= 2.0 ** -60
    got = orthogonalize(x)
    assert bool((got[0] == 0).all())
    assert bool(got[1].isnan().all()) and bool(got[2].isnan().all())
    assert t.equal(got[4], clean[4])
    check(x[3], got[3])
    assert bool((orthogonalize(x[:1], eps=0.0) == 0).all())


def test_empty_stacks():
    t = _t()
    from pretraining_optimizer_b200 import orthogonalize
    for shape in ((0, 4, 8), (2, 0, 8), (2, 4, 0)):
        x = t.empty(shape, dtype=t.bfloat16, device="cuda:0")
        assert orthogonalize(x).shape == shape


def test_the_same_bits_on_any_stream_and_in_a_graph():
    t = _t()
    from pretraining_optimizer_b200 import operator_status, orthogonalize
    rng = np.random.default_rng(12)
    x = t.from_numpy(_spectrum(rng, 24, 128, 1024, "plain")).to("cuda:0", t.bfloat16)
    odd = t.from_numpy(_spectrum(rng, 3, 24, 331, "plain")).to("cuda:0", t.bfloat16)
    first, first_odd = orthogonalize(x), orthogonalize(odd)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    for _ in range(3):   # two calls at once
        a, b = orthogonalize(x), orthogonalize(x, stream=side)
        c, d = orthogonalize(odd), orthogonalize(odd, stream=side)
        t.cuda.synchronize()
        assert t.equal(a, first) and t.equal(b, first) and t.equal(c, first_odd) and t.equal(d, first_odd)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        g1, g2 = orthogonalize(x), orthogonalize(odd)
    x2 = t.from_numpy(_spectrum(rng, 24, 128, 1024, "plain")).to("cuda:0", t.bfloat16)
    x.copy_(x2)
    graph.replay()
    t.cuda.synchronize()
    assert t.equal(g1, orthogonalize(x2)) and t.equal(g2, first_odd)
    operator_status()


def test_agrees_with_the_step_on_one_head():
    """A [128, c] weight as MuonH sees it and as a stack of one: the same Newton-Schulz output, up to the
    step's own 16-bit operands (held to 1e-2 in its tests) and the rounding of the stack's result."""
    t = _t()
    from pretraining_optimizer_b200 import MuonH, orthogonalize
    rng = np.random.default_rng(13)
    g = t.from_numpy(_spectrum(rng, 1, 128, 512, "plain")[0]).to("cuda:0", t.bfloat16)
    w = t.from_numpy(0.02 * rng.standard_normal((128, 512))).to("cuda:0", t.float32)
    opt = MuonH([w], beta=0.0, nesterov=False)
    opt.step([g.float()], 0.01)
    step = opt.update(0).double()
    opt.close()
    got = orthogonalize(g).double()
    assert float((got - step).norm() / step.norm()) <= 1e-2 + 2.0 ** -8


@pytest.mark.parametrize("shape", [(700, 16, 40), (600, 100, 130), (40, 128, 512), (20, 64, 1024), (70, 600, 65), (1, 16, 41000),
                                   (1, 41000, 16), (2, 128, 5000)])
def test_stacks_of_every_size(shape):
    """Several matrices per SM (with the late start), clusters of 2, 4 and 8, and long sides of many accumulations."""
    t = _t()
    from pretraining_optimizer_b200 import operator_status, orthogonalize
    x = t.from_numpy(_spectrum(np.random.default_rng(14), *shape, "plain")).to("cuda:0", t.bfloat16)
    check(x, orthogonalize(x))
    operator_status()


def test_refusals_of_the_binding():
    t = _t()
    from pretraining_optimizer_b200 import MuonHError, orthogonalize
    x = t.zeros(2, 130, 200, dtype=t.bfloat16, device="cuda:0")
    with pytest.raises(MuonHError, match="128"):
        orthogonalize(x)
    x = x[:, :8]
    with pytest.raises(TypeError):
        orthogonalize(x.float())
    with pytest.raises(ValueError):
        orthogonalize(x[None])
    with pytest.raises(ValueError):
        orthogonalize(x.mT)
    with pytest.raises(ValueError):
        orthogonalize(x, out=t.zeros(2, 8, 199, dtype=t.bfloat16, device="cuda:0"))
    with pytest.raises(TypeError):
        orthogonalize(x, out=t.zeros(2, 8, 200, dtype=t.float16, device="cuda:0"))
    with pytest.raises(ValueError):
        orthogonalize(x, out=x[:1].expand(2, 8, 200))
    with pytest.raises(MuonHError):
        orthogonalize(x, ns_steps=17)
