"""Cases and plain forms of the 8-bit linear layer's operators and layer norm.

A GPT's linear layers between two Muon steps: layer norm, the product in
8-bit floating point with a scale for each block of 128, the gradient with
respect to its input, the weight's gradient from the 8-bit activation that
the forward pass kept (what the Muon step takes), and layer norm's backward
pass.  ``own`` false: elementary torch operations; true: the library's
kernels.

The 8-bit tensor: e4m3 values, row-major, the row length rounded up to 128
with zeros; each block of R x 128 (R = 1 or 128) has a scale 2^e, the byte
e + 127, with e the smallest integer >= -117 such that the block's largest
magnitude is at most 448 * 2^e.
"""
import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "fp8": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp32": 4, "fp8": 1}


def listed():
    return [
        # one token behind its last layer norm: the smallest call
        {"name": "norm_1x768", "kind": "norm", "rows": 1, "n": 0, "k": 768, "x": "bf16", "out": "bf16"},
        # the residual stream kept in fp32, a batch of 16 x 1024 tokens
        {"name": "norm_16384x1280_fp32", "kind": "norm", "rows": 16384, "n": 0, "k": 1280, "x": "fp32", "out": "bf16"},
        # a training batch's backward pass through a wide layer norm
        {"name": "norm_back_8192x4096", "kind": "norm_back", "rows": 8192, "n": 0, "k": 4096, "x": "bf16", "out": "bf16"},
        # the same from an activation kept in 8 bits, a ragged batch
        {"name": "norm_back_4099x1280_fp8", "kind": "norm_back", "rows": 4099, "n": 0, "k": 1280, "x": "fp8", "out": "bf16"},
        # one token through the MLP's up projection: bound by the weights
        {"name": "linear_1x5120x1280", "kind": "linear", "rows": 1, "n": 5120, "k": 1280, "x": "fp8", "out": "bf16"},
        # a square projection of a training batch
        {"name": "linear_8192x4096x4096", "kind": "linear", "rows": 8192, "n": 4096, "k": 4096, "x": "fp8", "out": "bf16"},
        # the largest up projection: 16 sequences of 1024 tokens
        {"name": "linear_16384x16384x4096", "kind": "linear", "rows": 16384, "n": 16384, "k": 4096, "x": "fp8", "out": "bf16"},
        # layer norm written in 8 bits straight into a projection, a small model
        {"name": "norm_linear_2048x768x768", "kind": "norm_linear", "rows": 2048, "n": 768, "k": 768, "x": "bf16", "out": "bf16"},
        # the gradient that goes back through the up projection, a ragged batch
        {"name": "input_grad_4099x1280x5120", "kind": "input_grad", "rows": 4099, "n": 5120, "k": 1280, "x": "bf16", "out": "bf16"},
        # the weight gradient of a wide projection
        {"name": "weight_grad_8192x4096x4096", "kind": "weight_grad", "rows": 8192, "n": 4096, "k": 4096, "x": "fp8", "out": "fp32"},
        # many tokens, a small and oddly sized matrix: few tiles, a long sum
        {"name": "weight_grad_16384x768x1003", "kind": "weight_grad", "rows": 16384, "n": 768, "k": 1003, "x": "fp8", "out": "fp32"},
        # an activation stored in 8 bits and read back
        {"name": "checkpoint_8192x5120", "kind": "checkpoint", "rows": 8192, "n": 0, "k": 5120, "x": "bf16", "out": "bf16"},
    ]


def draw(rng):
    def spread(lo, hi):  # even over the logarithm
        return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))

    def dim(lo, hi):  # a layer's width: a multiple of 128, of 8, or any number
        d = spread(lo, hi)
        step = rng.choice((128, 128, 8, 1))
        return max(lo, d // step * step)

    kind = rng.choice(("norm", "norm_back", "linear", "norm_linear", "input_grad", "weight_grad", "checkpoint"))
    case = {"kind": kind, "rows": spread(1, 16384), "n": 0, "k": dim(128, 8192), "x": "bf16", "out": "bf16"}
    if kind in ("norm", "checkpoint"):
        case["x"] = rng.choice(("bf16", "fp32"))
    if kind == "norm":
        case["out"] = rng.choice(("bf16", "fp32"))
    if kind == "norm_back":
        case["x"], case["out"] = rng.choice((("bf16", "bf16"), ("fp32", "fp32"), ("fp8", "bf16"), ("fp8", "fp32")))
    if kind in ("linear", "norm_linear", "input_grad", "weight_grad"):
        case["n"] = dim(128, 8192)
        # the norm's result is rounded to 8 bits: its product says nothing in 32
        case["out"] = "bf16" if kind == "norm_linear" else rng.choice(("bf16", "fp32"))
    if kind in ("linear", "weight_grad"):
        case["x"] = "fp8"
    return case


# ------------------------------------------------------------ inputs


def _blocks(x, block_rows):
    """x padded with zeros to whole blocks, as (row blocks, R, column blocks, 128)."""
    r, c = x.shape
    x = torch.nn.functional.pad(x, (0, -c % 128, 0, -r % block_rows))
    return x.view(x.shape[0] // block_rows, block_rows, x.shape[1] // 128, 128)


def _pow2(e):
    """2 ** e of whole numbers -126 <= e <= 127, from the exponent bits: exp2 and ldexp may be a unit off."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _to8(x, block_rows):
    """(e4m3 values, scale bytes) of a 2-D tensor of 32 or 64 bits."""
    b = _blocks(x, block_rows)
    f, e = torch.frexp(b.abs().nan_to_num(0.0, 0.0).amax((1, 3)))
    e = torch.where(f > 0.875, e - 8, e - 9)  # 448 = 0.875 * 2^9
    e = torch.where(f == 0, torch.full_like(e, -117), e.clamp(min=-117))
    q = (b * _pow2(-e)[:, None, :, None]).float()
    q = torch.where(q.isfinite(), q, torch.full_like(q, float("nan"))).to(torch.float8_e4m3fn)
    q = q.view(b.shape[0] * block_rows, -1)[: x.shape[0]].contiguous()
    scale = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, -e.shape[1] % 4))
    return q, scale.contiguous()


def _values(q, scale, cols, block_rows, dtype=torch.float32):
    """The numbers that an 8-bit tensor stands for."""
    s = _pow2(scale.int() - 127)[:, : q.shape[1] // 128].to(dtype)
    s = s.repeat_interleave(block_rows, 0)[: q.shape[0]]
    return (q.to(dtype).view(q.shape[0], -1, 128) * s[:, :, None]).view(q.shape[0], -1)[:, :cols]


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _activations(g, rows, k):
    """A residual stream: tokens of unequal size, a few columns far larger than the others."""
    x = _randn(g, rows, k) * torch.exp(0.3 * _randn(g, rows, 1))
    return x * torch.exp2(6.0 * (torch.rand(k, generator=g, device="cuda") > 0.99)) + 0.1


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    rows, n, k, kind = case["rows"], case["n"], case["k"], case["kind"]
    s = dict(case)
    if kind in ("norm", "norm_linear", "norm_back", "checkpoint"):
        x = _activations(g, rows, k)
        if kind == "norm_back":
            x64 = x.double()
            s["mean"] = x64.mean(1).float()
            s["rstd"] = (x64.var(1, correction=0) + EPS).rsqrt().float()
            s["dy"] = (1e-3 * _randn(g, rows, k)).to(TYPES[case["out"]])
        s["x"] = _to8(x, 1) if case["x"] == "fp8" else x.to(TYPES[case["x"]])
        s["weight"] = 1.0 + 0.1 * _randn(g, k)
        s["bias"] = 0.1 * _randn(g, k)
    if kind in ("linear", "weight_grad"):
        s["x"] = _to8(_activations(g, rows, k), 1)
    if kind in ("linear", "norm_linear"):
        s["w"] = _to8(0.02 * _randn(g, n, k), 128)
    if kind == "input_grad":
        s["w"] = _to8(0.02 * _randn(g, k, n), 128)  # the transposed copy of the weights
    if kind in ("input_grad", "weight_grad"):
        s["dy"] = (1e-3 * _randn(g, rows, n) * torch.exp(_randn(g, rows, 1))).bfloat16()
    return s


# ------------------------------------------------------------ plain forms


def _norm(x, w, b):
    mean = x.mean(1, keepdim=True)
    rstd = (x - mean).square().mean(1, keepdim=True).add(EPS).rsqrt()
    return (x - mean) * rstd * w + b, mean[:, 0], rstd[:, 0]


def _plain(s):
    kind, n, k, out = s["kind"], s["n"], s["k"], TYPES[s["out"]]
    if kind == "norm":
        y, mean, rstd = _norm(s["x"].float(), s["weight"], s["bias"])
        return y.to(out), mean, rstd
    if kind == "norm_back":
        dy = s["dy"].float()
        x = _values(*s["x"], k, 1) if isinstance(s["x"], tuple) else s["x"].float()
        xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
        g = dy * s["weight"]
        dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        return dx.to(out), (dy * xh).sum(0), dy.sum(0)
    if kind == "linear":
        return (_values(*s["x"], k, 1) @ _values(*s["w"], k, 128).t()).to(out)
    if kind == "norm_linear":  # the norm in 64 bits: its result is rounded to 8
        y, mean, rstd = _norm(s["x"].double(), s["weight"].double(), s["bias"].double())
        y = _values(*_to8(y, 1), k, 1)
        return (y @ _values(*s["w"], k, 128).t()).to(out), mean.float(), rstd.float()
    if kind == "input_grad":
        dy = _values(*_to8(s["dy"].float(), 1), n, 1)
        return (dy @ _values(*s["w"], n, 128).t()).to(out)
    if kind == "weight_grad":
        return (s["dy"].float().t() @ _values(*s["x"], k, 1)).to(out)
    return _values(*_to8(s["x"].float(), 1), k, 1).to(out)  # checkpoint


def _own(s):
    import muon_newton_schulz_step_amd as muon

    kind, n, k, out = s["kind"], s["n"], s["k"], TYPES[s["out"]]
    if kind == "norm":
        return muon.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, out_dtype=out)
    if kind == "norm_back":
        x = muon.Tensor8(*s["x"], k) if isinstance(s["x"], tuple) else s["x"]
        return muon.layer_norm_backward(s["dy"], x, s["weight"], s["mean"], s["rstd"])
    if kind == "linear":
        return muon.matmul8(muon.Tensor8(*s["x"], k), muon.Tensor8(*s["w"], k, block_rows=128), out_dtype=out)
    if kind == "norm_linear":
        y, mean, rstd = muon.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, out_dtype=TYPES["fp8"])
        return muon.matmul8(y, muon.Tensor8(*s["w"], k, block_rows=128), out_dtype=out), mean, rstd
    if kind == "input_grad":
        return muon.matmul8(muon.quantize8(s["dy"]), muon.Tensor8(*s["w"], n, block_rows=128), out_dtype=out)
    if kind == "weight_grad":
        return muon.weight_grad(s["dy"], muon.Tensor8(*s["x"], k), out_dtype=out)
    return muon.dequantize8(muon.quantize8(s["x"]), dtype=out)  # checkpoint


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    rows, n, k, kind = case["rows"], case["n"], case["k"], case["kind"]
    x, out = SIZE[case["x"]], SIZE[case["out"]]
    if kind == "norm":
        return {"bytes": rows * k * (x + out) + 8 * rows + 8 * k, "flops": 8 * rows * k}
    if kind == "norm_back":  # dy and dx have the output's type
        return {"bytes": rows * k * (x + 2 * out) + 8 * rows + 12 * k, "flops": 14 * rows * k}
    if kind == "checkpoint":  # the 8-bit copy is written and read too
        return {"bytes": rows * k * (x + 2 + out), "flops": 3 * rows * k}
    if kind == "linear":
        return {"bytes": rows * k + n * k + out * rows * n, "flops": 2 * rows * n * k}
    if kind == "norm_linear":  # the 8-bit activation is an output: it is kept for the backward pass
        return {"bytes": rows * k * (x + 1) + n * k + out * rows * n, "flops": 2 * rows * n * k}
    if kind == "input_grad":
        return {"bytes": rows * n * x + n * k + out * rows * k, "flops": 2 * rows * n * k}
    return {"bytes": rows * n * 2 + rows * k + out * n * k, "flops": 2 * rows * n * k}  # weight_grad


# ------------------------------------------------------------ 64 bits


def _two_to(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round8(v, rows):
    """The values that `v` has after rounding to e4m3 in blocks of rows x 128, by arithmetic in 64 bits."""
    r, c = v.shape
    t = torch.zeros(-(-r // rows) * rows, -(-c // 128) * 128, dtype=torch.float64, device=v.device)
    t[:r, :c] = v
    t = t.reshape(t.shape[0] // rows, rows, -1, 128)
    top = t.abs().amax(3, keepdim=True).amax(1, keepdim=True)
    unit = _two_to(torch.ceil(torch.log2((top / 448).clamp(min=2.0 ** -117)) - 1e-12).clamp(min=-117))
    unit = torch.where(top > 448 * unit, 2 * unit, unit)
    unit = torch.where((top <= 224 * unit) & (unit > 2.0 ** -117), unit / 2, unit)
    t = t / unit
    mag = torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6)) + 1e-14)
    step = _two_to(mag - 3)
    t = torch.round(t / step) * step * unit
    return t.reshape(t.shape[0] * rows, -1)[:r, :c]


def _read8(pair, rows, cols):
    """An 8-bit tensor's values in 64 bits."""
    q, s = pair
    r = torch.arange(q.shape[0], device=q.device) // rows
    c = torch.arange(cols, device=q.device) // 128
    return q[:, :cols].double() * _two_to(s.to(torch.int64) - 127)[r][:, c]


def exact(case, seed):
    s = prepare(case, seed)
    kind, n, k = case["kind"], case["n"], case["k"]
    if kind in ("norm", "norm_linear"):
        x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
        mean = x.sum(1) / k
        var = (x * x).sum(1) / k - mean * mean
        rstd = 1.0 / torch.sqrt(var + EPS)
        y = torch.addcmul(b, (x - mean[:, None]) * rstd[:, None], w)
        if kind == "norm_linear":
            y = torch.mm(_round8(y, 1), _read8(s["w"], 128, k).t().contiguous())
        return y, mean, rstd
    if kind == "norm_back":
        dy, w, r = s["dy"].double(), s["weight"].double(), s["rstd"].double()
        x = _read8(s["x"], 1, k) if case["x"] == "fp8" else s["x"].double()
        xh = (x - s["mean"].double()[:, None]) * r[:, None]
        a, c = torch.mv(dy, w) / k, torch.mv(dy * xh, w) / k
        dx = r[:, None] * (dy * w[None, :] - a[:, None] - c[:, None] * xh)
        return dx, torch.einsum("tc,tc->c", dy, xh), dy.sum(0)
    if kind == "linear":
        return torch.mm(_read8(s["x"], 1, k), _read8(s["w"], 128, k).t().contiguous())
    if kind == "input_grad":
        return torch.mm(_round8(s["dy"].double(), 1), _read8(s["w"], 128, n).t().contiguous())
    if kind == "weight_grad":
        return torch.mm(s["dy"].double().t().contiguous(), _read8(s["x"], 1, k))
    return _round8(s["x"].double(), 1)
