"""The 8-bit integer linear path and its layer norm, case by case: what is computed, on which inputs, and its plain form.

Operators (`nvfp4_block_scaled_18_b200`):
  quantize       nvfp4_i8_quantize            one scale for each row (token, or output channel of a weight)
  layernorm      nvfp4_layernorm              forward, with the statistics that the backward pass reads
  backward       nvfp4_layernorm_backward     gradients of the input, of the gain and of the bias
  norm_quantize  nvfp4_layernorm_i8_quantize  layer norm, and its result in 8 bits, in one pass
  gemm           nvfp4_i8_gemm                8-bit product with a scale for each token and each channel

8-bit codes are whole numbers, so both forms take the same steps in fp32, each rounded once:
  quantize   amax = max|x|; scale = amax / 127; code = rint(x * (127 / amax)); amax < 2^-110 gives scale 0 and codes 0
  layernorm  mean = sum(x) / K and var = sum((x - mean)^2) / K with sums in 64 bits, mean and rstd = 1 / sqrt(var + eps)
             rounded to fp32; y = ((x - mean) * rstd) * gain + bias
"""
import math

import torch

own = False

EPS = 1e-5
BF16, F32 = "bf16", "f32"
TYPES = {BF16: torch.bfloat16, F32: torch.float32}
LARGEST = 8192 * 28672 * 8192          # products of the largest 8-bit linear listed


def listed():
    return [
        # one token of a decode step: latency
        dict(name="quantize one token", op="quantize", rows=1, cols=4096, dtype=BF16, gap=0),
        # the input of a down projection over a whole prompt: bandwidth
        dict(name="quantize prompt", op="quantize", rows=8192, cols=14336, dtype=BF16, gap=0),
        # a decode step of 16 sequences whose residual stream is kept in fp32
        dict(name="layernorm decode", op="layernorm", rows=16, cols=5120, dtype=F32, params=F32, gap=0),
        # a training batch's forward pass: bf16 activations, fp32 gain and bias
        dict(name="layernorm batch", op="layernorm", rows=8192, cols=4096, dtype=BF16, params=F32, gap=0),
        # a short ragged batch's backward pass
        dict(name="backward short batch", op="backward", rows=333, cols=5120, dtype=BF16, params=BF16, gap=0),
        # a training batch's backward pass, wide rows, everything in fp32
        dict(name="backward batch", op="backward", rows=8192, cols=8192, dtype=F32, params=F32, gap=0),
        # the input of an 8-bit linear for four tokens in flight
        dict(name="norm_quantize decode", op="norm_quantize", rows=4, cols=5120, dtype=BF16, params=BF16, gap=0),
        # the same over a prompt whose rows are part of a wider buffer
        dict(name="norm_quantize prompt", op="norm_quantize", rows=2048, cols=4096, dtype=BF16, params=BF16, gap=64),
        # one token: the weight is read once
        dict(name="gemm one token", op="gemm", rows=1, out=14336, cols=4096, dtype=BF16, bias=True),
        # 61 sequences of a serving batch into the down projection
        dict(name="gemm serving batch", op="gemm", rows=61, out=5120, cols=27648, dtype=BF16, bias=False),
        # a ragged chunk of a prompt, fp32 output
        dict(name="gemm prompt chunk", op="gemm", rows=777, out=11008, cols=4096, dtype=F32, bias=True),
        # a whole prompt through the largest projection
        dict(name="gemm prompt", op="gemm", rows=8192, out=28672, cols=8192, dtype=BF16, bias=False),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over the logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("quantize", "layernorm", "backward", "norm_quantize", "gemm", "gemm"))
    if op == "gemm":
        rows, out, cols = _spread(rng, 1, 8192), _spread(rng, 64, 28672), 16 * _spread(rng, 4, 1792)
        cols = max(16, min(cols, LARGEST // (rows * out) // 16 * 16))
        return dict(op=op, rows=rows, out=out, cols=cols, dtype=rng.choice((BF16, F32)), bias=rng.random() < 0.5)
    case = dict(op=op, rows=_spread(rng, 1, 8192), cols=16 * _spread(rng, 4, 896), dtype=rng.choice((BF16, F32)),
                gap=rng.choice((0, 0, 64)))
    if op != "quantize":
        case["params"] = F32 if case["dtype"] == F32 else rng.choice((BF16, F32))
    return case


def _matrix(rows, cols, dtype, gap):
    return torch.empty((rows, cols + gap), dtype=dtype, device="cuda")[:, :cols]


def _rows_in_8_bits(x):
    """Codes and scales of every row: the quantizer's plain form."""
    x = x.float()
    amax = x.abs().amax(dim=1, keepdim=True)
    of = torch.full_like(amax, 127.0)
    zero = amax < 2.0 ** -110
    scale = torch.where(zero, 0.0, amax / of)
    inv = torch.where(zero, 0.0, of / amax)
    return torch.round(x * inv).to(torch.int8), scale.squeeze(1)


def _normed(x, gain, bias):
    """Layer norm's plain form before its last rounding, and its statistics."""
    x = x.float()
    mean = x.double().mean(dim=1, keepdim=True).float()
    d = x - mean
    var = d.double().square().mean(dim=1, keepdim=True)
    rstd = (1.0 / torch.sqrt(var + EPS)).float()
    return d * rstd * gain.float() + bias.float(), mean.squeeze(1), rstd.squeeze(1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, rows, cols, dtype = case["op"], case["rows"], case["cols"], TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def activations(gap):
        """Normal values, one channel in a hundred 50 times larger, a shift for each channel; the last of many rows is
        empty padding."""
        x = normal(rows, cols)
        x[:, torch.randperm(cols, generator=g, device="cuda")[:max(1, cols // 100)]] *= 50.0
        if op != "quantize":
            x += 0.5 * normal(cols)
        if rows >= 64:
            x[-1] = 0.0
        to = _matrix(rows, cols, dtype, gap)
        return to.copy_(x)

    s = dict(op=op)
    if op == "gemm":
        out = case["out"]
        s["a"], s["a_scales"] = _rows_in_8_bits(activations(0))
        s["w"], s["w_scales"] = _rows_in_8_bits(0.02 * normal(out, cols))
        s["bias"] = normal(out) if case["bias"] else None
        s["y"] = _matrix(rows, out, dtype, 0)
        return s
    gap = case["gap"]
    s["x"] = activations(gap)
    if op in ("quantize", "norm_quantize"):
        s["codes"] = _matrix(rows, cols, torch.int8, 0)
        s["scales"] = torch.empty(rows, device="cuda")
    if op != "quantize":
        s["gain"] = (1.0 + 0.2 * normal(cols)).to(TYPES[case["params"]])
        s["bias"] = (0.1 * normal(cols)).to(TYPES[case["params"]])
    if op == "layernorm":
        s["y"] = _matrix(rows, cols, dtype, gap)
        s["mean"], s["rstd"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    if op == "backward":
        s["dy"] = _matrix(rows, cols, dtype, gap).copy_(0.01 * normal(rows, cols))
        _, s["mean"], s["rstd"] = _normed(s["x"], s["gain"], s["bias"])
        s["dx"] = _matrix(rows, cols, dtype, gap)
        s["dgain"], s["dbias"] = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    return s


def _run_own(s):
    import nvfp4_block_scaled_18_b200 as nv
    op = s["op"]
    if op == "quantize":
        nv.nvfp4_i8_quantize(s["x"], s["codes"], s["scales"])
        return s["codes"], s["scales"]
    if op == "layernorm":
        nv.nvfp4_layernorm(s["x"], s["y"], s["gain"], s["bias"], eps=EPS, mean=s["mean"], rstd=s["rstd"])
        return s["y"], s["mean"], s["rstd"]
    if op == "backward":
        if "workspace" not in s:          # kept with the layer
            s["workspace"] = nv.LayerNormWorkspace(*s["x"].shape)
        nv.nvfp4_layernorm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["dx"], s["gain"], dgamma=s["dgain"],
                                    dbeta=s["dbias"], workspace=s["workspace"])
        return s["dx"], s["dgain"], s["dbias"]
    if op == "norm_quantize":
        nv.nvfp4_layernorm_i8_quantize(s["x"], s["codes"], s["scales"], s["gain"], s["bias"], eps=EPS)
        return s["codes"], s["scales"]
    nv.nvfp4_i8_gemm(s["a"], s["a_scales"], s["w"], s["w_scales"], s["y"], bias=s["bias"])
    return s["y"]


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "quantize":
        return _rows_in_8_bits(s["x"])
    if op == "layernorm":
        y, mean, rstd = _normed(s["x"], s["gain"], s["bias"])
        return y.to(s["x"].dtype), mean, rstd
    if op == "backward":
        x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
        xhat = (x - s["mean"][:, None]) * rstd
        dz = dy * s["gain"].float()
        dx = rstd * (dz - dz.mean(dim=1, keepdim=True) - xhat * (dz * xhat).mean(dim=1, keepdim=True))
        return dx.to(s["x"].dtype), (dy * xhat).sum(dim=0), dy.sum(dim=0)
    if op == "norm_quantize":
        return _rows_in_8_bits(_normed(s["x"], s["gain"], s["bias"])[0])
    y = (s["a"].float() @ s["w"].float().T) * s["a_scales"][:, None] * s["w_scales"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["y"].dtype)


def work(case):
    rows, cols, size = case["rows"], case["cols"], 2 if case["dtype"] == BF16 else 4
    n = rows * cols
    if case["op"] == "gemm":
        out = case["out"]
        return {"bytes": n + out * cols + rows * out * size + 4 * (rows + out + (out if case["bias"] else 0)),
                "flops": 2 * rows * out * cols}
    if case["op"] == "quantize":
        return {"bytes": n * (size + 1) + 4 * rows, "flops": 4 * n}
    params = cols * (2 if case["params"] == BF16 else 4)
    if case["op"] == "layernorm":
        return {"bytes": 2 * n * size + 2 * params + 8 * rows, "flops": 8 * n}
    if case["op"] == "backward":
        return {"bytes": 3 * n * size + params + 8 * cols + 8 * rows, "flops": 14 * n}
    return {"bytes": n * (size + 1) + 2 * params + 4 * rows, "flops": 12 * n}


def exact(case, seed):
    """The definitions in 64 bits. A code next to a border has no value apart from the steps in fp32: None for codes."""
    s = prepare(case, seed)
    op = s["op"]
    if op == "gemm":
        y = torch.matmul(s["a"].double(), s["w"].double().t())
        y *= torch.outer(s["a_scales"].double(), s["w_scales"].double())
        return y if s["bias"] is None else y.add_(s["bias"].double())
    x = s["x"].double()
    if op == "quantize":
        return None, x.abs().max(dim=1).values / 127.0
    gain, bias = s["gain"].double(), s["bias"].double()
    if op == "backward":
        # through the definition y = gain * xhat + bias with the given statistics: mean depends on x by 1/K and rstd by
        # -rstd^3 (x - mean) / K, so dL/dx = sum of the three terms
        mean, rstd, dy = s["mean"].double().unsqueeze(1), s["rstd"].double().unsqueeze(1), s["dy"].double()
        centred = x - mean
        to_hat = dy * gain
        by_rstd = torch.einsum("rc,rc->r", to_hat, centred).unsqueeze(1)
        by_mean = -(to_hat.sum(1, keepdim=True) * rstd)
        dx = to_hat * rstd + by_mean / case["cols"] - by_rstd * rstd ** 3 * centred / case["cols"]
        return dx, torch.einsum("rc,rc->c", dy, centred * rstd), torch.einsum("rc->c", dy)
    var, mean = torch.var_mean(x, dim=1, correction=0)
    rstd = torch.rsqrt(var + EPS)
    y = torch.addcmul(bias, gain, (x - mean.unsqueeze(1)) * rstd.unsqueeze(1))
    if op == "layernorm":
        return y, mean, rstd
    return None, y.abs().max(dim=1).values / 127.0
