"""The operators where their rows lie more than 32 bits apart, and where two
threads call them at once: the same bits as from compact tensors, one at a time."""
import threading

import pytest
import torch

from pretraining_optimizer_b200 import (block_matmul, block_quantize, block_quantize_weight, layer_norm,
                                        layer_norm_backward, operator_status, orthogonalize)

pytestmark = pytest.mark.gpu

FAR = 2 ** 31 + 64   # elements between rows


def _randn(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def _apart(x):
    """x's values in a view whose first dimension steps by FAR elements."""
    inner = x[0].numel()
    buffer = torch.empty(FAR * (x.shape[0] - 1) + inner, dtype=x.dtype, device="cuda")
    view = buffer.as_strided(x.shape, (FAR, *x.stride()[1:]))
    view.copy_(x)
    return view


def _equal(got, want):
    for a, b in zip(got, want, strict=True):
        assert (a is None) == (b is None)
        if a is not None:
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# within a warp, in the ring, and wider than a block holds
@pytest.mark.parametrize("n", (200, 2048, 9000))
def test_norm_of_rows_far_apart(n):
    x, dy, w, b = _randn(1, 3, n).bfloat16(), _randn(2, 3, n).bfloat16(), _randn(3, n), _randn(4, n)
    y, mean, rstd = layer_norm(x, w, b)
    want = layer_norm_backward(dy, x, w, mean, rstd, bias=True)
    far = _apart(x)
    _equal(layer_norm(far, w, b), (y, mean, rstd))
    _equal(layer_norm_backward(dy, far, w, mean, rstd, bias=True), want)
    layer_norm(far, w, b, out=far)
    _equal((far,), (y,))
    far.copy_(dy)
    _equal(layer_norm_backward(far, x, w, mean, rstd, bias=True), want)
    operator_status()


def test_products_of_rows_far_apart():
    x = _randn(1, 3, 200).bfloat16()
    a, b = block_quantize(x), block_quantize(_randn(2, 70, 200))
    want = block_matmul(*a, *b)
    out = _apart(torch.zeros_like(want))
    _equal(block_quantize(out.copy_(want), columns=True), block_quantize(want, columns=True))
    out.zero_()
    block_matmul(*a, *b, out=out)
    _equal((out,), (want,))
    del out
    q = _apart(a[0].contiguous().view(torch.uint8)).view(torch.float8_e4m3fn)
    scale = _apart(a[1])
    _equal((block_matmul(q, scale, *b), block_matmul(*b, q, scale)), (want, block_matmul(*b, *a)))
    operator_status()


# TMA reads and writes the aligned one; the odd width goes through the scratch
@pytest.mark.parametrize("cols", (264, 203))
def test_orthogonalize_matrices_far_apart(cols):
    x = _randn(1, 3, 32, cols).bfloat16()
    want = orthogonalize(x)
    far = _apart(x)
    _equal((orthogonalize(far),), (want,))
    orthogonalize(far, out=far)
    _equal((far,), (want,))
    operator_status()


def test_two_threads_at_once():
    def work(seed):
        x, w = _randn(seed, 500, 512).bfloat16(), _randn(seed + 10, 300, 512)
        y, mean, rstd = layer_norm(x, w[0].contiguous())
        dx, dw, _ = layer_norm_backward(x, y, w[0].contiguous(), mean, rstd)
        z = block_matmul(*block_quantize(y), *block_quantize_weight(w)[:2])
        return y, dx, dw, z, orthogonalize(x.view(4, 125, 512))

    want = [work(seed) for seed in range(2)]
    torch.cuda.synchronize()
    failed = []

    def run(seed):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got = work(seed)
                    torch.cuda.current_stream().synchronize()
                    _equal(got, want[seed])
        except BaseException as e:   # an assertion in a thread would be lost
            failed.append(e)

    threads = [threading.Thread(target=run, args=(seed,)) for seed in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    operator_status()
