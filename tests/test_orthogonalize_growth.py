"""Which runs orthogonalize keeps in fp16 pairs: the others ask for fp64 scratch; and that its tests' bound tells
pairs from single operands, by emulation of the kernel's roundings (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import pretraining_optimizer_b200 as P
from oracle import operators as O
from pretraining_optimizer_b200.muonh import OrthogonalizeDesc

A = 0x10000   # an address that is never read
CUBIC = (1.5, -0.5, 0.0)


def _scratch(steps, coeffs=P.QUINTIC, batch=2, rows=32, cols=64):
    d = OrthogonalizeDesc(A, A, batch, rows, cols, rows * cols, cols, rows * cols, cols, 1, steps, *coeffs, 1e-7)
    return P.library().muonh_orthogonalize_workspace(ctypes.byref(d))


def test_runs_that_pairs_hold():
    assert all(_scratch(n) == 0 for n in range(6)) and all(_scratch(n) > 0 for n in range(6, 17))
    # 1.5^15 = 438, 1.5^16 = 657; 1.875^9 = 286, 1.875^10 = 537
    assert _scratch(15, CUBIC) == 0 and _scratch(16, CUBIC) > 0
    assert _scratch(9, (1.875, -1.25, 0.375)) == 0 and _scratch(10, (1.875, -1.25, 0.375)) > 0
    # factors below one, iterates that leave the range, and factors beyond any range
    assert _scratch(2, (0.5, 0.25, 0.0)) > 0 and _scratch(3, (20.0, -40.0, 21.0)) > 0
    assert _scratch(1, (1.0, 3.0, 0.0)) > 0 and _scratch(16, (1e30, 1e30, 1e30)) > 0
    assert _scratch(0, (0.0, 0.0, 0.0)) == 0


def test_scratch_is_bounded():
    matrix = 128 * 2048 * 8 + 5 * 128 * 128 * 8
    assert _scratch(6, batch=1, rows=128, cols=2048) >= matrix
    assert _scratch(6, batch=896, rows=128, cols=2048) <= 2 ** 28
    assert _scratch(6, batch=2 ** 24, rows=1, cols=1) <= 2 ** 28
    # sizes that the call refuses, and whose products do not fit in 64 bits
    assert _scratch(6, batch=2 ** 62) == _scratch(6, rows=4, cols=2 ** 62) == _scratch(6, rows=2 ** 62, cols=4) == 0
    # one matrix at least, however long
    assert 2 ** 30 * 8 <= _scratch(6, batch=3, rows=1, cols=2 ** 30) <= 2 ** 30 * 8 + 2 ** 20


def _rounded(x, dtype, scale, parts):
    """x 2^scale as a sum of `parts` numbers of the type, scaled back."""
    left, total = np.ldexp(x, scale), 0.0
    for _ in range(parts):
        part = torch.from_numpy(left).to(dtype).double().numpy()
        total, left = total + part, left - part
    return np.ldexp(total, -scale)


def _emulate(x, dtype, parts):
    """Five default steps on the r x r matrices of x with operands of `parts` fp16 numbers each (Q in the end: of
    the type), fp32 results, and the power-of-two scales that fill fp16's range."""
    a, b, c = O.QUINTIC
    fp32 = lambda v: v.astype(np.float32).astype(np.float64)  # noqa: E731
    norm = np.linalg.norm(x) + 1e-7
    gram, q = fp32(x @ x.T / norm ** 2), None
    for k in range(5):
        g = _rounded(gram, torch.float16, 15, parts)
        p = fp32(a * np.eye(len(g)) + b * gram + c * fp32(g @ g))
        p16 = _rounded(p, torch.float16, 14, parts)
        q = p if q is None else fp32(_rounded(q, torch.float16, (14, 12, 10, 8)[k - 1], parts) @ p16)
        gram = fp32(_rounded(fp32(g @ p16), torch.float16, 15, parts) @ p16)
    return _rounded(q, dtype, 6 if dtype == torch.float16 else 0, parts) @ x / norm


@pytest.mark.parametrize("name", ["bf16", "fp16"])
@pytest.mark.parametrize("kind", ["exact1", "exact4", "8+1e-3", "1+1e-2"])
def test_the_bound_tells_pairs_from_single_operands(kind, name):
    from test_gpu_orthogonalize_growth import PAIRS, matrices
    dtype = {"bf16": torch.bfloat16, "fp16": torch.float16}[name]
    for shape in ((128, 512), (64, 64)):
        x = torch.from_numpy(matrices(kind, 1, *shape)[0]).to(dtype).double().numpy()
        ref = O.orthogonalize(x[None])[0]
        size = np.linalg.norm(ref)
        half = torch.finfo(dtype).eps / 2
        assert np.linalg.norm(_emulate(x, dtype, 2) - ref) <= PAIRS[name] * size
        # beyond the bound and the rounding of the result together, or overflowed to NaN
        with np.errstate(all="ignore"):
            assert not np.linalg.norm(_emulate(x, dtype, 1) - ref) <= 2 * (PAIRS[name] + half) * size
