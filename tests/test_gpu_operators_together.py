"""The operators as one training step uses them together (B200 only): a normed,
block-quantised linear layer forward and backward, its weight stepped by MuonH and
its norm's weight by AdamW, the new weight quantised, and the same gradient
orthogonalised head by head.  Every stage is held to fp64 on what it was given."""
import numpy as np
import pytest

import oracle
from oracle import aux, operators as O
from test_gpu_block import check_product, check_quantized
from test_gpu_norm import check_backward, check_forward
from test_gpu_orthogonalize import check as check_orthogonal

pytestmark = pytest.mark.gpu

TOKENS, INPUTS, HEADS, HEAD = 300, 256, 4, 64
OUTPUTS = HEADS * HEAD


def _values(q, s):
    return O.block_values(q.float().cpu().numpy(), s.cpu().numpy())


def test_two_training_steps():
    import torch
    import pretraining_optimizer_b200 as P
    dev = torch.device("cuda:0")
    rng = np.random.default_rng(21)

    def draw(*shape, scale=1.0, dtype=torch.float32):
        return torch.from_numpy(scale * rng.standard_normal(shape)).to(dev, dtype)

    w = draw(OUTPUTS, INPUTS, scale=0.02)
    gain = 1 + draw(INPUTS, scale=0.1)
    m, v = torch.zeros_like(gain), torch.zeros_like(gain)
    target = draw(TOKENS, OUTPUTS, scale=0.1)
    opt = P.MuonH([w])
    radius = oracle.radius(w.double().cpu().numpy())
    momentum = np.zeros((OUTPUTS, INPUTS))
    grad = torch.empty_like(w)
    for step in (1, 2):
        x = draw(TOKENS, INPUTS, dtype=torch.bfloat16)
        wq, ws, wt, wts = P.block_quantize_weight(w)
        check_quantized(w, wq, ws, 128)
        # forward
        y, _, rstd = P.layer_norm(x, gain, rms=True, eps=1e-6)
        check_forward(x, gain, None, 1e-6, True, y, None, rstd)
        yq, ys, yt, yts = P.block_quantize(y, columns=True)
        out = P.block_matmul(yq, ys, wq, ws)
        check_product(_values(yq, ys), _values(wq, ws), out, INPUTS)
        # backward of half the squared distance to the target, in two halves of the batch that add up
        dout = (out.float() - target).to(torch.bfloat16)
        grad.zero_()
        gq, gs = P.block_quantize(dout)
        dy = P.block_matmul(gq, gs, wt, wts)
        check_product(_values(gq, gs), _values(wt, wts), dy, OUTPUTS)
        want, size = 0.0, 0.0
        for rows in (slice(0, 128), slice(128, TOKENS)):
            gt, gts = P.block_quantize(dout[rows], rows=False, columns=True)
            yt, yts = P.block_quantize(y[rows], rows=False, columns=True)
            P.block_matmul(gt, gts, yt, yts, out=grad, accumulate=True)
            want = want + _values(gt, gts) @ _values(yt, yts).T
            size = size + np.abs(_values(gt, gts)) @ np.abs(_values(yt, yts)).T
        # at most 2 x 2 blocks of 128, four MMAs each, as the products' own tests count them
        assert np.all(np.abs(grad.double().cpu().numpy() - want) <= (16 * 2.0 ** -22 + 2.0 ** -23) * size)
        dx, dgain, _ = P.layer_norm_backward(dy, x, gain, None, rstd)
        check_backward(dy, x, gain, None, rstd, dx, dgain, None)
        # one update per head, beside the whole matrix's
        heads = grad.unflatten(0, (HEADS, HEAD)).to(torch.bfloat16)
        check_orthogonal(heads, P.orthogonalize(heads))
        # the optimizers read those gradients
        before, g64 = w.double().cpu().numpy(), grad.double().cpu().numpy()
        gain_before, m_before, v_before = (t.double().cpu().numpy() for t in (gain, m, v))
        opt.step([grad], 0.01)
        w_ref, momentum, _, _ = oracle.muonh_step(before, momentum, g64, 0.01, radius)
        assert np.linalg.norm(w.double().cpu().numpy() - w_ref) <= 1e-4 * radius
        P.adamw_step([gain], [m], [v], [dgain], step, 1e-3)
        ref, _, _ = aux.adamw_step(gain_before, m_before, v_before, dgain.double().cpu().numpy(), step, 1e-3)
        assert np.allclose(gain.double().cpu().numpy(), ref, rtol=0, atol=1e-6)
    opt.device_status()
    P.operator_status()
    opt.close()


def test_a_captured_backward_and_update():
    """The backward half and the update captured in one graph and replayed on new activations."""
    import torch
    import pretraining_optimizer_b200 as P
    dev = torch.device("cuda:0")
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(200, 256, generator=g, device=dev).bfloat16()
    dout = torch.randn(200, 128, generator=g, device=dev).bfloat16()
    w0 = 0.02 * torch.randn(128, 256, generator=g, device=dev)
    new_x = torch.randn(200, 256, generator=g, device=dev).bfloat16()

    def backward(w, grad):
        _, _, wt, wts = P.block_quantize_weight(w)
        _, _, rstd = P.layer_norm(x, rms=True)
        q, s, qt, st = P.block_quantize(dout, columns=True)
        xt, xts = P.block_quantize(x, rows=False, columns=True)
        P.block_matmul(qt, st, xt, xts, out=grad)
        dx, _, _ = P.layer_norm_backward(P.block_matmul(q, s, wt, wts), x, None, None, rstd)
        return dx

    results = []
    for captured in (False, True):
        w, grad = w0.clone(), torch.empty_like(w0)
        opt = P.MuonH([w], groups=1)
        args = opt.step_args([grad], 0.01)
        kept = x.clone()
        if captured:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                dx = backward(w, grad)
                opt.step_device(args)
            graph.replay()
            x.copy_(new_x)
            graph.replay()
        else:
            backward(w, grad)
            opt.step_device(args)
            x.copy_(new_x)
            dx = backward(w, grad)
            opt.step_device(args)
        torch.cuda.synchronize()
        results.append((w.clone(), grad.clone(), dx.clone()))
        x.copy_(kept)
        opt.close()
    for a, b in zip(*results):
        assert torch.equal(a, b)
    P.operator_status()
