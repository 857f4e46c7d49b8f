"""The fp64 oracle of the operators around the update, against independent computations (no GPU)."""
import numpy as np
import pytest
import torch

import oracle
from oracle import operators as O


def test_e4m3_matches_the_cast_of_every_bf16_value():
    bits = np.arange(1 << 16, dtype=np.uint16)
    x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).double()
    x = x[torch.isfinite(x) & (x.abs() <= 448)]
    ref = x.float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.e4m3(x.numpy()), ref)


def test_e4m3_ties_go_to_even():
    assert O.e4m3([1.0625, 1.1875, -1.0625, 2.0 ** -10, 3 * 2.0 ** -10, 448.0]).tolist() == \
        [1.0, 1.25, -1.0, 0.0, 2.0 ** -8, 448.0]


def test_block_exponents_are_the_smallest_that_hold_the_block():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((130, 300)) * np.exp(4 * rng.standard_normal((130, 1)))
    x[:, 128:256] *= (np.arange(130) % 3 > 0)[:, None]
    for rows in (1, 128):
        k = O.block_exponents(x, rows)
        top = np.abs(x) / np.ldexp(448.0, O.spread(k, rows, *x.shape))
        assert np.all(top <= 1)
        for i in range(k.shape[0]):
            for j in range(k.shape[1]):
                block = np.abs(x[i * rows:(i + 1) * rows, 128 * j:128 * (j + 1)]).max()
                assert (block == 0 and k[i, j] == 0) or block > np.ldexp(448.0, k[i, j] - 1)
    assert O.block_exponents(np.array([[2.0 ** -140]]), 1)[0, 0] == -127
    assert O.block_exponents(np.array([[448.0], [448.5], [896.0]]), 1).ravel().tolist() == [0, 1, 1]


def test_quantised_values_are_within_half_a_step():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((40, 200))
    q, s = O.block_quantize(x, 1)
    back = O.block_values(q, s)
    # e4m3 rounds to 2^-4 relative, or half of 2^-9 times the scale below its normal values
    step = np.ldexp(2.0 ** -10, O.spread(s.astype(np.int64) - 127, 1, *x.shape))
    assert np.all(np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), step))


@pytest.mark.parametrize("rms", [False, True])
def test_layer_norm_and_its_gradients_match_autograd(rms):
    g = torch.Generator().manual_seed(2)
    x, dy = (torch.randn(7, 33, generator=g, dtype=torch.float64) for _ in range(2))
    w, b = (torch.randn(33, generator=g, dtype=torch.float64) for _ in range(2))
    for t in (x, w, b):
        t.requires_grad_(True)
    mean = torch.zeros(7, 1, dtype=torch.float64) if rms else x.mean(1, keepdim=True)
    rstd = ((x - mean).square().mean(1, keepdim=True) + 1e-5).rsqrt()
    y = (x - mean) * rstd * w + b
    if not rms:
        assert torch.allclose(y, torch.nn.functional.layer_norm(x, (33,), w, b), atol=1e-12)
    y.backward(dy)
    n = lambda t: t.detach().numpy()  # noqa: E731
    got, m, r = O.layer_norm(n(x), n(w), n(b), 1e-5, rms)
    assert np.allclose(got, n(y), atol=1e-12)
    dx, dw, db = O.layer_norm_backward(n(dy), n(x), n(w), m, r, rms)
    assert np.allclose(dx, n(x.grad), atol=1e-12) and np.allclose(dw, n(w.grad), atol=1e-12)
    assert np.allclose(db, n(b.grad), atol=1e-12)


@pytest.mark.parametrize("shape", [(3, 8, 20), (2, 20, 8), (1, 1, 5)])
def test_orthogonalize_matches_the_steps_newton_schulz(shape):
    x = np.random.default_rng(3).standard_normal(shape)
    got = O.orthogonalize(x)
    for i in range(shape[0]):
        ref = oracle.newton_schulz(x[i])
        assert np.allclose(got[i], ref, atol=1e-12)
