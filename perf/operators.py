"""The operators around one weight update, as calls a training program makes.

    norm            layer norm or RMS norm of rows of activations, forward
    norm_backward   its gradients: of the activations, and of the weight and
                    bias, which AdamW trains
    linear          a linear layer's forward pass in 8-bit floating point with a
                    scale for each block of 128 (activations quantised in the
                    call, weights quantised once after the update)
    linear_backward the gradients of its activations and of its weight, the fp32
                    matrix that MuonH's step reads
    weights         quantising an updated fp32 weight in both orientations
    orthogonalize   the Newton-Schulz iteration over a stack of matrices with a
                    small side: one update per attention head

`run` computes a case in plain torch operations, or with `own` set through this
repository's entry points.  Sizes follow the Qwen3 tables of the synthetic sets
(d_model 2048, d_ff 6144; heads of 128, per layer 16 for queries and 8 each for
keys and values).
"""
import math

import torch

own = False

GROUP = 128          # elements that share one 8-bit scale
FP8_MAX = 448.0      # the largest e4m3 value
COEFFS = (3.4445, -4.7750, 2.0315)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the final norm of one position: the smallest call, latency only
        dict(name="norm_one_row", op="norm", rows=1, n=2048, dtype="bf16", rms=True, bias=False),
        # a layer's input norm over one microbatch of 2 x 4096 tokens
        dict(name="norm_layer", op="norm", rows=8192, n=2048, dtype="bf16", rms=False, bias=True),
        # the q norm's gradient: 16 heads of 8192 tokens, a weight of 128 summed over 131072 rows
        dict(name="norm_backward_heads", op="norm_backward", rows=131072, n=128, dtype="bf16", rms=True, bias=False),
        # an odd width in fp32: nothing is aligned, and rows are few
        dict(name="norm_backward_odd", op="norm_backward", rows=1021, n=5003, dtype="fp32", rms=False, bias=True),
        # a short ragged batch through a projection whose sizes are not multiples of 128
        dict(name="linear_ragged", op="linear", tokens=77, inputs=1000, outputs=520, dtype="fp16"),
        # the gate projection's forward pass over one microbatch
        dict(name="linear_gate", op="linear", tokens=8192, inputs=2048, outputs=6144, dtype="bf16"),
        # ... and both of its gradients
        dict(name="linear_backward_gate", op="linear_backward", tokens=8192, inputs=2048, outputs=6144, dtype="bf16"),
        # that projection's weight after an update
        dict(name="weights_gate", op="weights", inputs=2048, outputs=6144),
        # a few small updates with an odd side
        dict(name="orthogonalize_small", op="orthogonalize", batch=5, rows=33, cols=200, tall=False, strided=False,
             dtype="bf16"),
        # the query, key and value heads of one layer
        dict(name="orthogonalize_layer", op="orthogonalize", batch=32, rows=128, cols=2048, tall=False, strided=False,
             dtype="bf16"),
        # an output projection's heads: column blocks of one matrix, with a head size below 128
        dict(name="orthogonalize_output", op="orthogonalize", batch=16, rows=96, cols=2048, tall=True, strided=True,
             dtype="fp16"),
        # the query, key and value heads of 28 layers
        dict(name="orthogonalize_model", op="orthogonalize", batch=896, rows=128, cols=2048, tall=False, strided=False,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "linear", "linear_backward", "weights", "orthogonalize", "orthogonalize"])
    if op in ("norm", "norm_backward"):
        n = _log(rng, 16, 16384) if rng.random() < 0.5 else 16 * _log(rng, 1, 1024)
        return dict(op=op, rows=_log(rng, 1, max(1, min(131072, (1 << 25) // n))), n=n,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), rms=rng.random() < 0.5, bias=rng.random() < 0.5)
    if op in ("linear", "linear_backward"):
        inputs, outputs = _log(rng, 64, 4096), _log(rng, 64, 6144)
        if rng.random() < 0.5:
            inputs, outputs = -(-inputs // 128) * 128, -(-outputs // 128) * 128
        return dict(op=op, tokens=_log(rng, 1, max(1, min(8192, (8192 * 2048 * 6144) // (inputs * outputs)))),
                    inputs=inputs, outputs=outputs, dtype=rng.choice(["bf16", "bf16", "fp16"]))
    if op == "weights":
        return dict(op=op, inputs=_log(rng, 64, 6144), outputs=_log(rng, 64, 6144))
    rows = rng.choice([128, 64, _log(rng, 1, 128)])
    cols = _log(rng, rows, 8192) if rng.random() < 0.5 else 64 * max(-(-rows // 64), _log(rng, 1, 128))
    return dict(op=op, batch=_log(rng, 1, max(1, min(896, (896 * 128 * 2048) // (128 * cols)))), rows=rows, cols=cols,
                tall=rng.random() < 0.4, strided=rng.random() < 0.4, dtype=rng.choice(["bf16", "bf16", "fp16"]))


# ----------------------------------------------------------------- the inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, rows, n):
    """Activations: channels of different sizes, a few of them outliers, and a mean that is not zero."""
    channel = torch.exp(0.5 * _randn(g, n))
    channel[: max(1, n // 256)] *= 20.0
    return _randn(g, rows, n).mul_(channel).add_(0.3 * channel)


def _gradients(g, rows, n):
    """Gradients of activations: small, and of very different sizes from token to token."""
    return _randn(g, rows, n).mul_(1e-3 * torch.exp(_randn(g, rows, 1)))


def _padded(rows, cols, dtype):
    """An uninitialised rows x cols matrix whose row stride is a multiple of 16 elements."""
    return torch.empty(rows, -(-cols // 16) * 16, dtype=dtype, device="cuda")[:, :cols]


def _kept(q):
    out = _padded(*q.shape, torch.float8_e4m3fn)
    out.copy_(q)
    return out


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    state = dict(case)
    if op in ("norm", "norm_backward"):
        rows, n, dtype = case["rows"], case["n"], DTYPES[case["dtype"]]
        state["x"] = _activations(g, rows, n).to(dtype)
        state["weight"] = 1.0 + 0.1 * _randn(g, n)
        state["shift"] = 0.1 * _randn(g, n) if case["bias"] else None
        if op == "norm_backward":
            state["dy"] = _gradients(g, rows, n).to(dtype)
            _, state["mean"], state["rstd"] = _norm(state["x"].float(), state["weight"], None, case["rms"])
    elif op in ("linear", "linear_backward"):
        tokens, inputs, outputs, dtype = case["tokens"], case["inputs"], case["outputs"], DTYPES[case["dtype"]]
        x = _activations(g, tokens, inputs).to(dtype)
        w = 0.02 * _randn(g, outputs, inputs)
        if op == "linear":  # kept since the weight's last update
            q, s = _quantize_blocks(w)
            state.update(x=x, w=_kept(q), w_scale=s)
        else:  # kept since the update and since the forward pass
            q, s = _quantize_blocks(w.t().contiguous())
            xt, xt_scale = _quantize_rows(x.float().t().contiguous())
            state.update(dy=_gradients(g, tokens, outputs).to(dtype), wt=_kept(q), wt_scale=s, xt=_kept(xt), xt_scale=xt_scale)
    elif op == "weights":
        state["w"] = 0.02 * _randn(g, case["outputs"], case["inputs"])
    else:
        batch, rows, cols = case["batch"], case["rows"], case["cols"]
        if case["tall"]:
            rows, cols = cols, rows
        # an update in earnest: noise over a few strong directions
        r = max(1, min(4, case["rows"]))
        x = _randn(g, batch, rows, cols).add_(torch.matmul(_randn(g, batch, rows, r), _randn(g, batch, r, cols))).mul_(1e-3)
        x = x.to(DTYPES[case["dtype"]])
        if case["strided"]:  # heads as column blocks of one matrix
            whole = x.transpose(0, 1).reshape(rows, batch * cols)
            x = whole.unflatten(1, (batch, cols)).transpose(0, 1)
        state["x"] = x
    return state


# ------------------------------------------------------------ the plain forms

def _norm(x, weight, shift, rms, eps=1e-6):
    mean = None if rms else x.mean(-1)
    centred = x if rms else x - mean[..., None]
    rstd = torch.rsqrt(centred.square().mean(-1) + eps)
    y = centred * rstd[..., None] * weight
    return (y if shift is None else y + shift), mean, rstd


def _norm_backward(dy, x, weight, mean, rstd):
    unit = (x if mean is None else x - mean[..., None]) * rstd[..., None]
    inner = dy * weight
    dx = inner - unit * (inner * unit).mean(-1, keepdim=True)
    if mean is not None:
        dx = dx - inner.mean(-1, keepdim=True)
    return dx * rstd[..., None], (dy * unit).sum(0), dy.sum(0)


def _exponent(amax):
    """The smallest k with amax <= 448 * 2^k, at least -127; 0 for a block of zeros."""
    mantissa, e = torch.frexp(amax)  # 448 = 0.875 * 2^9
    k = torch.where(mantissa <= 0.875, e - 9, e - 8).clamp_(min=-127)
    return torch.where(amax > 0, k, torch.zeros_like(k))


def _blocks(x, height):
    """x (fp32) padded and split into blocks of height x 128: [rows, height, columns, 128]."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, -cols % GROUP, 0, -rows % height))
    return x.view(x.shape[0] // height, height, x.shape[1] // GROUP, GROUP)


def _quantize(x, height):
    b = _blocks(x, height)
    k = _exponent(b.abs().amax(dim=(1, 3)))
    q = torch.ldexp(b, -k[:, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(b.shape[0] * height, -1)[: x.shape[0], : x.shape[1]], (k + 127).to(torch.uint8)


def _quantize_rows(x):
    return _quantize(x, 1)


def _quantize_blocks(w):
    return _quantize(w, GROUP)


def _values(q, scale, dtype=torch.float32):
    """What a quantised matrix stands for; its scales are one row for each of its rows, or one for each 128 of them."""
    rows, cols = q.shape
    s = torch.ldexp(torch.ones((), dtype=dtype, device=q.device), scale.to(torch.int32) - 127)
    s = s.repeat_interleave(GROUP, 1)[:, :cols]
    if scale.shape[0] != rows:
        s = s.repeat_interleave(GROUP, 0)[:rows]
    return q.to(dtype) * s


def _newton_schulz(x, steps=5, eps=1e-7):
    a, b, c = COEFFS
    y = x.mT if x.shape[-2] > x.shape[-1] else x
    y = y / (y.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    for _ in range(steps):
        gram = y @ y.mT
        y = a * y + (b * gram + c * (gram @ gram)) @ y
    return y.mT if x.shape[-2] > x.shape[-1] else y


# -------------------------------------------------------------------- the run

def run(state):
    op = state["op"]
    if own:
        import pretraining_optimizer_b200 as P

        if op == "norm":
            return P.layer_norm(state["x"], state["weight"], state["shift"], eps=1e-6, rms=state["rms"])
        if op == "norm_backward":
            return P.layer_norm_backward(state["dy"], state["x"], state["weight"], state["mean"], state["rstd"],
                                         bias=state["bias"])
        if op == "linear":
            q, s = P.block_quantize(state["x"])
            return P.block_matmul(q, s, state["w"], state["w_scale"], dtype=state["x"].dtype)
        if op == "linear_backward":
            q, s, qt, st = P.block_quantize(state["dy"], columns=True)
            return (P.block_matmul(q, s, state["wt"], state["wt_scale"], dtype=state["dy"].dtype),
                    P.block_matmul(qt, st, state["xt"], state["xt_scale"], dtype=torch.float32))
        if op == "weights":
            return P.block_quantize_weight(state["w"])
        return P.orthogonalize(state["x"])

    if op == "norm":
        y, mean, rstd = _norm(state["x"].float(), state["weight"], state["shift"], state["rms"])
        return y.to(state["x"].dtype), mean, rstd
    if op == "norm_backward":
        dx, dw, db = _norm_backward(state["dy"].float(), state["x"].float(), state["weight"], state["mean"], state["rstd"])
        return dx.to(state["x"].dtype), dw, db if state["bias"] else None
    if op == "linear":
        x = _values(*_quantize_rows(state["x"].float()))
        return (x @ _values(state["w"], state["w_scale"]).t()).to(state["x"].dtype)
    if op == "linear_backward":
        dy = state["dy"].float()
        dx = _values(*_quantize_rows(dy)) @ _values(state["wt"], state["wt_scale"]).t()
        dw = _values(*_quantize_rows(dy.t().contiguous())) @ _values(state["xt"], state["xt_scale"]).t()
        return dx.to(state["dy"].dtype), dw
    if op == "weights":
        q, s = _quantize_blocks(state["w"])
        return q, s, q.t().contiguous(), s.t().contiguous()
    return _newton_schulz(state["x"].float()).to(state["x"].dtype)


# ------------------------------------------------------------------- the work

def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}[case.get("dtype", "fp32")]
    if op in ("norm", "norm_backward"):
        rows, n = case["rows"], case["n"]
        stats = 4 * rows * (1 if case["rms"] else 2)
        if op == "norm":
            return {"bytes": 2 * rows * n * size + 4 * n * (2 if case["bias"] else 1) + stats, "flops": 8 * rows * n}
        return {"bytes": 3 * rows * n * size + 4 * n * (3 if case["bias"] else 2) + stats, "flops": 14 * rows * n}
    if op in ("linear", "linear_backward"):
        m, k, n = case["tokens"], case["inputs"], case["outputs"]
        if op == "linear":
            return {"bytes": size * m * (k + n) + n * k, "flops": 2 * m * n * k}
        return {"bytes": size * m * (k + n) + n * k + m * k + 4 * n * k, "flops": 4 * m * n * k}
    if op == "weights":
        return {"bytes": 6 * case["inputs"] * case["outputs"], "flops": 2 * case["inputs"] * case["outputs"]}
    b, r, c = case["batch"], case["rows"], case["cols"]
    # one Gram product, the five steps on r x r matrices (17 products of them), one product with the matrix
    return {"bytes": 2 * size * b * r * c, "flops": b * (4 * r * r * c + 17 * 2 * r * r * r)}


# ------------------------------------------------- the definitions, in 64 bits

def _exact_quantized(x, height):
    """The values that quantising x in blocks of height x 128 keeps, its e4m3 values and its exponents, in 64 bits."""
    rows, cols = x.shape
    up, left = -(-rows // height), -(-cols // GROUP)
    whole = torch.zeros(up * height, left * GROUP, dtype=torch.float64, device=x.device)
    whole[:rows, :cols] = x.double()
    tiles = whole.reshape(up, height, left, GROUP)
    top = tiles.abs().amax(3).amax(1)
    k = torch.ceil(torch.log2(torch.where(top > 0, top, torch.full_like(top, FP8_MAX)) / FP8_MAX))
    # the logarithm may have been rounded across a border
    k = torch.where(top > FP8_MAX * torch.exp2(k), k + 1, k)
    k = torch.where((top > 0) & (top <= FP8_MAX * torch.exp2(k - 1)), k - 1, k)
    k = k.clamp(min=-127.0)
    v = tiles * torch.exp2(-k)[:, None, :, None]
    # e4m3: three bits behind the leading one, exponents down to 2^-6; ties to even
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    v = torch.round(v / step) * step
    kept = v.reshape(up * height, -1)[:rows, :cols]
    real = (v * torch.exp2(k)[:, None, :, None]).reshape(up * height, -1)[:rows, :cols]
    return real, kept, k


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = state["x"].double()
        mean = x.mean(1)
        if not case["rms"]:
            x = x - mean[:, None]
        rstd = 1.0 / torch.sqrt((x * x).sum(1) / x.shape[1] + 1e-6)
        y = x * rstd[:, None] * state["weight"].double()[None, :]
        if state["shift"] is not None:
            y = y + state["shift"].double()[None, :]
        return y, (None if case["rms"] else mean), rstd
    if op == "norm_backward":
        dy, x, w, rstd = state["dy"].double(), state["x"].double(), state["weight"].double(), state["rstd"].double()[:, None]
        n = x.shape[1]
        if not case["rms"]:
            x = x - state["mean"].double()[:, None]
        xhat = x * rstd
        g = dy * w[None, :]
        dx = rstd * (g - (0.0 if case["rms"] else g.sum(1, keepdim=True) / n) - xhat * ((g * xhat).sum(1, keepdim=True) / n))
        return dx, torch.einsum("ij,ij->j", dy, xhat), (dy.sum(0) if case["bias"] else None)
    if op == "linear":
        x, _, _ = _exact_quantized(state["x"], 1)
        return torch.matmul(x, _values(state["w"], state["w_scale"], torch.float64).mT)
    if op == "linear_backward":
        rows, _, _ = _exact_quantized(state["dy"], 1)
        columns, _, _ = _exact_quantized(state["dy"].mT, 1)
        return (torch.matmul(rows, _values(state["wt"], state["wt_scale"], torch.float64).mT),
                torch.matmul(columns, _values(state["xt"], state["xt_scale"], torch.float64).mT))
    if op == "weights":
        _, q, _ = _exact_quantized(state["w"], GROUP)
        return q, None, q.mT.contiguous(), None
    x = state["x"].double()
    if case["tall"]:
        x = x.mT
    x = x / (torch.linalg.matrix_norm(x, keepdim=True) + 1e-7)
    a, b, c = COEFFS
    eye = torch.eye(x.shape[-2], dtype=torch.float64, device=x.device)
    for _ in range(5):
        gram = torch.matmul(x, x.mT)
        x = torch.matmul(a * eye + b * gram + c * torch.matmul(gram, gram), x)
    return (x.mT if case["tall"] else x).contiguous()
