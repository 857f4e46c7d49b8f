"""Which runs orthogonalize keeps in fp16 pairs: the others ask for fp64 scratch (no GPU)."""
import ctypes

import pretraining_optimizer_b200 as P
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
    # one matrix at least, however long
    assert 2 ** 30 * 8 <= _scratch(6, batch=3, rows=1, cols=2 ** 30) <= 2 ** 30 * 8 + 2 ** 20
