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
