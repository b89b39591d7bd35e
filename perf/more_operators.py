"""Cases and plain forms of a block's fused operators and of gradient clipping.

What stands between a GPT's linear layers, and between their gradients and the
Muon step: the 8-bit product with bias, activation and residual in its
epilogue, in bf16, fp32 or straight into the next product's 8 bits; its
backward pass up to the operands of the two gradient products; the norms
after and before a block fused with the block's gate and the residual stream's
scale; and the norm of all gradients with their clipping.  ``own`` false:
elementary torch operations; true: the library's kernels.

The 8-bit tensor: e4m3 values, row-major, the row length rounded up to 128
with zeros; each block of R x 128 (R = 1 or 128) has a scale 2^e, the byte
e + 127, with e the smallest integer >= -117 such that the block's largest
magnitude is at most 448 * 2^e.
"""
import math

import torch

own = False

EPS = 1e-5
CLIP_EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "fp8": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp32": 4, "fp8": 1, "none": 0}


def listed():
    return [
        # one token through the MLP's up projection: bound by the weights
        {"name": "linear_1x5120x1280_relu2", "kind": "linear", "rows": 1, "n": 5120, "k": 1280, "act": "relu2", "residual": "none", "out": "bf16"},
        # the down projection of a ragged batch, added to a residual stream kept in fp32
        {"name": "linear_4099x1280x5120_fp32", "kind": "linear", "rows": 4099, "n": 1280, "k": 5120, "act": "none", "residual": "fp32", "out": "fp32"},
        # a training batch through the whole MLP: up, squared ReLU, 8 bits, down, residual
        {"name": "mlp_4096x1280x5120_relu2", "kind": "mlp", "rows": 4096, "n": 5120, "k": 1280, "act": "relu2", "residual": "bf16", "out": "bf16"},
        # the largest: 16 sequences of 1024 tokens, a wide model with GELU
        {"name": "mlp_16384x4096x16384_gelu", "kind": "mlp", "rows": 16384, "n": 16384, "k": 4096, "act": "gelu", "residual": "bf16", "out": "bf16"},
        # back through the squared ReLU of a training batch, and its bias
        {"name": "linear_back_8192x5120_relu2", "kind": "linear_back", "rows": 8192, "n": 5120, "k": 0, "act": "relu2", "residual": "none", "out": "bf16"},
        # the same through a GELU of odd width, a short ragged batch
        {"name": "linear_back_1027x1003_gelu", "kind": "linear_back", "rows": 1027, "n": 1003, "k": 0, "act": "gelu", "residual": "none", "out": "bf16"},
        # one token between two blocks of a small model, RMS norms on both sides
        {"name": "norm_1x768_rms", "kind": "norm", "rows": 1, "k": 768, "x": "bf16", "branch": "bf16", "out": "bf16", "rms": True, "post": True, "gate": True, "scale": True},
        # a batch of 16 x 1024 tokens, the residual stream in fp32, its norm in 8 bits for the next product
        {"name": "norm_16384x1280_fp32_fp8", "kind": "norm", "rows": 16384, "k": 1280, "x": "fp32", "branch": "bf16", "out": "fp8", "rms": False, "post": False, "gate": True, "scale": True},
        # the backward pass of a wide model's batch with all that the operator has
        {"name": "norm_back_8192x4096", "kind": "norm_back", "rows": 8192, "k": 4096, "x": "bf16", "branch": "bf16", "out": "bf16", "rms": False, "post": True, "gate": True, "scale": True},
        # a ragged batch of a small model: residual sum and RMS norm alone, the stream in fp32
        {"name": "norm_back_4099x1280_rms", "kind": "norm_back", "rows": 4099, "k": 1280, "x": "fp32", "branch": "bf16", "out": "bf16", "rms": True, "post": False, "gate": False, "scale": False},
        # the gradients' norm of a small GPT, for the log: 8 layers of width 640
        {"name": "grad_norm_8x640", "kind": "clip", "layers": 8, "d": 640, "ff": 2560, "x": "bf16", "out": "none", "clipped": False},
        # fp32 accumulators of a wide GPT clipped into the bf16 gradients that the step takes
        {"name": "clip_4x4096_fp32", "kind": "clip", "layers": 4, "d": 4096, "ff": 16384, "x": "fp32", "out": "bf16", "clipped": True},
    ]


def draw(rng):
    def spread(lo, hi):  # even over the logarithm
        return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))

    def dim(lo, hi):  # a layer's width: a multiple of 128, of 8, or any number
        d = spread(lo, hi)
        step = rng.choice((128, 128, 8, 1))
        return max(lo, d // step * step)

    kind = rng.choice(("linear", "mlp", "linear_back", "norm", "norm_back", "clip"))
    if kind == "clip":
        d = dim(128, 2048)
        return {"kind": kind, "layers": spread(1, 12), "d": d, "ff": 4 * d, "x": rng.choice(("bf16", "fp32")),
                "out": rng.choice(("none", "bf16", "same")), "clipped": rng.choice((True, True, False))}
    case = {"kind": kind, "rows": spread(1, 16384), "k": 0 if kind == "linear_back" else dim(128, 4096 if kind == "mlp" else 8192)}
    if kind in ("linear", "mlp", "linear_back"):
        case["n"] = 4 * case["k"] if kind == "mlp" else dim(128, 8192)
        case["act"] = rng.choice(("none", "relu", "relu2", "gelu", "gelu_tanh", "silu")[kind != "linear":])
        case["out"] = "bf16" if kind == "linear_back" else rng.choice(("bf16", "bf16", "fp32"))
        case["residual"] = "none" if kind == "linear_back" else rng.choice(("none", "bf16", "fp32"))
        if kind == "mlp":  # the hidden layer is rounded to 8 bits: its product says nothing in 32
            case["out"] = "bf16"
    else:
        case["x"], case["branch"] = rng.choice((("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32")))
        case["out"] = case["branch"] if kind == "norm_back" else rng.choice(("bf16", "fp32", "fp8"))
        case["rms"], case["post"] = rng.random() < 0.5, rng.random() < 0.5
        case["gate"], case["scale"] = rng.random() < 0.5, rng.random() < 0.5
    return case


# ------------------------------------------------------------ inputs


def _pow2(e):
    """2 ** e of whole numbers -126 <= e <= 127, from the exponent bits: exp2 and ldexp may be a unit off."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _to8(x, block_rows):
    """(e4m3 values, scale bytes) of a 2-D tensor of 32 or 64 bits."""
    r, c = x.shape
    b = torch.nn.functional.pad(x, (0, -c % 128, 0, -r % block_rows))
    b = b.view(b.shape[0] // block_rows, block_rows, b.shape[1] // 128, 128)
    f, e = torch.frexp(b.abs().amax((1, 3)))
    e = torch.where(f > 0.875, e - 8, e - 9)  # 448 = 0.875 * 2^9
    e = torch.where(f == 0, torch.full_like(e, -117), e.clamp(min=-117))
    q = (b * _pow2(-e)[:, None, :, None]).float().to(torch.float8_e4m3fn)
    q = q.view(b.shape[0] * block_rows, -1)[:r].contiguous()
    scale = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, -e.shape[1] % 4))
    return q, scale.contiguous()


def _values(q, scale, cols, block_rows):
    """The numbers that an 8-bit tensor stands for."""
    s = _pow2(scale.int() - 127)[:, : q.shape[1] // 128]
    s = s.repeat_interleave(block_rows, 0)[: q.shape[0]]
    return (q.float().view(q.shape[0], -1, 128) * s[:, :, None]).view(q.shape[0], -1)[:, :cols]


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _activations(g, rows, k):
    """A residual stream: tokens of unequal size, a few columns far larger than the others."""
    x = _randn(g, rows, k) * torch.exp(0.3 * _randn(g, rows, 1))
    return x * torch.exp2(6.0 * (torch.rand(k, generator=g, device="cuda") > 0.99)) + 0.1


def _shapes(case):
    """A GPT's gradients: the matrices of each layer, and the gains and shifts of its two norms."""
    d, ff = case["d"], case["ff"]
    matrices = [(d, d), (d, d), (d, d), (d, d), (ff, d), (d, ff)] * case["layers"]
    return matrices, [(d,)] * (4 * case["layers"])


def _views(flat, shapes):
    """Tensors of the shapes, one behind the other in a flat buffer."""
    return [p.view(s) for p, s in zip(flat.split([math.prod(s) for s in shapes]), shapes)]


def _prepare_clip(case, g, s):
    matrices, vectors = _shapes(case)
    numbers = sum(map(math.prod, matrices)), sum(map(math.prod, vectors))
    big = (1e-3 * _randn(g, numbers[0])).to(TYPES[case["x"]])
    small = 1e-2 * _randn(g, numbers[1])  # the norms' gradients stay in fp32
    s["grads"] = _views(big, matrices) + _views(small, vectors)
    expected = math.sqrt(1e-6 * numbers[0] + 1e-4 * numbers[1])
    s["max_norm"] = 0.25 * expected if case["clipped"] else 4.0 * expected
    if case["out"] != "none":
        out = case["x"] if case["out"] == "same" else case["out"]
        s["flat"] = (torch.zeros(numbers[0], dtype=TYPES[out], device="cuda"), torch.zeros(numbers[1], device="cuda"))
        s["outs"] = _views(s["flat"][0], matrices) + _views(s["flat"][1], vectors)
    return s


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    s, kind = dict(case), case["kind"]
    if kind == "clip":
        return _prepare_clip(case, g, s)
    rows, k = case["rows"], case["k"]
    if kind in ("linear", "mlp"):
        n = case["n"]
        last = n if kind == "linear" else k
        s["x"] = _to8(_activations(g, rows, k), 1)
        s["w"] = _to8(0.02 * _randn(g, n, k), 128)
        s["bias"] = 0.1 * _randn(g, n)
        if kind == "mlp":
            s["w2"] = _to8(0.02 * _randn(g, k, n), 128)
            s["bias2"] = 0.1 * _randn(g, k)
        s["add"] = None if case["residual"] == "none" else _activations(g, rows, last).to(TYPES[case["residual"]])
        return s
    if kind == "linear_back":
        n = case["n"]
        s["z"] = (_randn(g, rows, n) * torch.exp(0.3 * _randn(g, rows, 1))).bfloat16()
        s["dy"] = (1e-3 * _randn(g, rows, n) * torch.exp(_randn(g, rows, 1))).bfloat16()
        return s
    s["x"] = _activations(g, rows, k).to(TYPES[case["x"]])
    s["b"] = (2.0 * _randn(g, rows, k) + 0.2).to(TYPES[case["branch"]])
    s["weight"], s["bias"] = 1.0 + 0.1 * _randn(g, k), 0.1 * _randn(g, k)
    s["pw"], s["pb"] = (1.0 + 0.1 * _randn(g, k), 0.1 * _randn(g, k)) if case["post"] else (None, None)
    s["g"] = 0.5 + 0.2 * _randn(g, k) if case["gate"] else None
    s["a"] = 0.9 + 0.05 * _randn(g, 1) if case["scale"] else None
    if case["rms"]:
        s["bias"] = s["pb"] = None
    if kind == "norm_back":  # what the forward pass kept, and the gradients that arrive
        r, _, s["stats"] = _norm_forward(s, torch.float64)
        s["r"], s["stats"] = r.to(TYPES[case["x"]]), s["stats"].float()
        s["dr"] = (1e-3 * _randn(g, rows, k)).to(TYPES[case["x"]])
        s["dh"] = (1e-3 * _randn(g, rows, k)).to(TYPES[case["branch"]])
    return s


# ------------------------------------------------------------ plain forms


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "relu2":
        return z.clamp(min=0.0) * z.clamp(min=0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "relu2":
        return 2.0 * z.clamp(min=0.0)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)
    s = 1.0 / (1.0 + torch.exp(-z))  # silu
    return s * (1.0 + z * (1.0 - s))


def _stats(x, rms):
    mean = torch.zeros_like(x[:, :1]) if rms else x.mean(1, keepdim=True)
    return mean, (x - mean).square().mean(1, keepdim=True).add(EPS).rsqrt()


def _norm_forward(s, dtype=torch.float32):
    """r = scale x + gate post(branch) and its norm, with both norms' statistics."""
    x, b = s["x"].to(dtype), s["b"].to(dtype)
    stats = torch.zeros(4, x.shape[0], dtype=dtype, device=x.device)
    if s["post"]:
        mean, rstd = _stats(b, s["rms"])
        stats[2], stats[3] = mean[:, 0], rstd[:, 0]
        b = (b - mean) * rstd * s["pw"] + (0.0 if s["pb"] is None else s["pb"])
    r = (x if s["a"] is None else s["a"] * x) + (b if s["g"] is None else s["g"] * b)
    mean, rstd = _stats(r, s["rms"])
    stats[0], stats[1] = mean[:, 0], rstd[:, 0]
    return r, (r - mean) * rstd * s["weight"] + (0.0 if s["bias"] is None else s["bias"]), stats


def _norm_plain(s):
    r, h, stats = _norm_forward(s)
    if s["out"] == "fp8":
        h = _values(*_to8(h, 1), s["k"], 1).bfloat16()
    else:
        h = h.to(TYPES[s["out"]])
    return r.to(s["x"].dtype), h, stats


def _norm_grad(g, xh, rstd, rms):
    """The gradient of a norm's input from that of its normalised row."""
    d = g - xh * (g * xh).mean(1, keepdim=True)
    return rstd * (d if rms else d - g.mean(1, keepdim=True))


def _norm_back_plain(s):
    st, rms = s["stats"][:, :, None], s["rms"]
    dh, r, b = s["dh"].float(), s["r"].float(), s["b"].float()
    rh = (r - st[0]) * st[1]
    d = s["dr"].float() + _norm_grad(dh * s["weight"], rh, st[1], rms)
    dx = d if s["a"] is None else s["a"] * d
    ds = None if s["a"] is None else (d.double() * s["x"].double()).sum().float().view(1)
    bh = (b - st[2]) * st[3] if s["post"] else b
    p = bh * s["pw"] + (0.0 if s["pb"] is None else s["pb"]) if s["post"] else bh
    dg = None if s["g"] is None else (d * p).sum(0)
    db = d if s["g"] is None else s["g"] * d
    dpw = dpb = None
    if s["post"]:
        dpw = (db * bh).sum(0)
        dpb = None if s["pb"] is None else db.sum(0)
        db = _norm_grad(db * s["pw"], bh, st[3], rms)
    dw, dbias = (dh * rh).sum(0), None if s["bias"] is None else dh.sum(0)
    return dx.to(s["x"].dtype), db.to(s["b"].dtype), dw, dbias, dpw, dpb, dg, ds


def _clip_plain(s):
    norm = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt()
    if s["out"] == "none":
        return norm.float()
    c = (s["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0).float()
    n = 6 * s["layers"]
    done = [(c * g.float()).to(o.dtype).view(-1) for g, o in zip(s["grads"], s["outs"])]
    return norm.float(), torch.cat(done[:n]), torch.cat(done[n:])


def _plain(s):
    kind = s["kind"]
    if kind == "clip":
        return _clip_plain(s)
    if kind == "norm":
        return _norm_plain(s)
    if kind == "norm_back":
        return _norm_back_plain(s)
    if kind == "linear_back":
        dz = s["dy"].float() * _act_grad(s["z"].float(), s["act"])
        return dz.bfloat16(), _values(*_to8(dz, 1), s["n"], 1).bfloat16(), dz.sum(0)
    n, k = s["n"], s["k"]
    z = _values(*s["x"], k, 1) @ _values(*s["w"], k, 128).t() + s["bias"]
    y = _act(z, s["act"])
    if kind == "mlp":
        y = _values(*_to8(y, 1), n, 1) @ _values(*s["w2"], n, 128).t() + s["bias2"]
    if s["add"] is not None:
        y = y + s["add"].float()
    y = y.to(TYPES[s["out"]])
    return (y, z.bfloat16()) if kind == "mlp" else y


def _own(s):
    import muon_newton_schulz_step_amd as muon

    kind, k = s["kind"], s["k"] if "k" in s else 0
    if kind == "clip":
        if s["out"] == "none":
            return muon.grad_norm(s["grads"])
        return muon.clip_grads(s["grads"], s["max_norm"], eps=CLIP_EPS, out=s["outs"]), *s["flat"]
    if kind == "norm":
        r, h, stats = muon.residual_norm(s["x"], s["b"], s["weight"], s["bias"], post_weight=s["pw"], post_bias=s["pb"],
                                         gate=s["g"], scale=s["a"], rms=s["rms"], eps=EPS, out_dtype=TYPES[s["out"]])
        return r, muon.dequantize8(h) if s["out"] == "fp8" else h, stats
    if kind == "norm_back":
        return tuple(muon.residual_norm_backward(s["dr"], s["dh"], s["r"], s["b"], s["weight"], s["stats"], x=s["x"],
                                                 bias=s["bias"] is not None, post_weight=s["pw"], post_bias=s["pb"],
                                                 gate=s["g"], scale=s["a"], rms=s["rms"]))
    act = None if s["act"] == "none" else s["act"]
    if kind == "linear_back":
        dz, dz8, dbias = muon.linear8_backward(s["dy"], s["z"], activation=act)
        return dz, muon.dequantize8(dz8), dbias
    x, w = muon.Tensor8(*s["x"], k), muon.Tensor8(*s["w"], k, block_rows=128)
    if kind == "linear":
        return muon.linear8(x, w, s["bias"], activation=act, residual=s["add"], out_dtype=TYPES[s["out"]])
    hidden, z = muon.linear8(x, w, s["bias"], activation=act, keep=True, out_dtype=torch.float8_e4m3fn)
    w2 = muon.Tensor8(*s["w2"], s["n"], block_rows=128)
    return muon.linear8(hidden, w2, s["bias2"], residual=s["add"], out_dtype=TYPES[s["out"]]), z


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    kind = case["kind"]
    if kind == "clip":  # the norm of all comes before the first clipped number: two readings, but one that is needed
        m, v = (sum(map(math.prod, t)) for t in _shapes(case))
        out = 0 if case["out"] == "none" else SIZE[case["x"] if case["out"] == "same" else case["out"]]
        return {"bytes": m * (SIZE[case["x"]] + out) + v * (4 + (4 if out else 0)), "flops": (2 + (1 if out else 0)) * (m + v)}
    rows, k = case["rows"], case["k"]
    if kind == "linear":
        n = case["n"]
        return {"bytes": rows * k + n * k + 4 * n + rows * n * (SIZE[case["out"]] + SIZE[case["residual"]]), "flops": 2 * rows * n * k}
    if kind == "mlp":  # the hidden layer is kept for the backward pass, in 8 bits and before the activation
        n = case["n"]
        return {"bytes": rows * k + 2 * n * k + 4 * (n + k) + rows * n * 3 + rows * k * (SIZE[case["out"]] + SIZE[case["residual"]]), "flops": 4 * rows * n * k}
    if kind == "linear_back":  # dy, z, dz; the 8-bit copy is written, read and given as values
        return {"bytes": rows * case["n"] * (2 + 2 + 2 + 2 + 2) + 4 * case["n"], "flops": 12 * rows * case["n"]}
    x, b = SIZE[case["x"]], SIZE[case["branch"]]
    vectors = 4 * k * (2 + 2 * case["post"] + case["gate"])
    if kind == "norm":
        out = 4 if case["out"] == "fp8" else SIZE[case["out"]]
        return {"bytes": rows * k * (2 * x + b + out) + 16 * rows + vectors, "flops": rows * k * (9 + 8 * case["post"])}
    # dr, dh, r, dx, dbranch; the branch itself for its norm and its gate, x for its scale
    moved = x * 3 + b * 2 + (b if case["post"] or case["gate"] else 0) + (x if case["scale"] else 0)
    return {"bytes": rows * k * moved + 16 * rows + 2 * vectors, "flops": rows * k * (16 + 16 * case["post"])}


# ------------------------------------------------------------ 64 bits


def _two_to(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round8(v):
    """The values that `v` has after rounding to e4m3 in blocks of 1 x 128, by arithmetic in 64 bits."""
    r, c = v.shape
    t = torch.zeros(r, -(-c // 128) * 128, dtype=torch.float64, device=v.device)
    t[:, :c] = v
    t = t.view(r, -1, 128)
    top = t.abs().amax(2, keepdim=True)
    unit = _two_to(torch.ceil(torch.log2((top / 448).clamp(min=2.0 ** -117)) - 1e-12).clamp(min=-117))
    unit = torch.where(top > 448 * unit, 2 * unit, unit)
    unit = torch.where((top <= 224 * unit) & (unit > 2.0 ** -117), unit / 2, unit)
    t = t / unit
    step = _two_to(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6)) + 1e-14) - 3)
    return (torch.round(t / step) * step * unit).view(r, -1)[:, :c]


def _read8(pair, rows, cols):
    """An 8-bit tensor's values in 64 bits."""
    q, s = pair
    r = torch.arange(q.shape[0], device=q.device) // rows
    c = torch.arange(cols, device=q.device) // 128
    return q[:, :cols].double() * _two_to(s.to(torch.int64) - 127)[r][:, c]


def _phi(z):
    """The normal distribution's function and density."""
    return torch.special.ndtr(z), torch.exp(-z * z / 2) * 0.3989422804014327


def _bend(z, act):
    """An activation and its slope."""
    if act in ("relu", "relu2"):
        on = torch.relu(z)
        return (on, (z > 0).double()) if act == "relu" else (on * on, 2 * on)
    if act == "gelu":
        below, density = _phi(z)
        return z * below, below + z * density
    if act == "silu":
        gate = torch.sigmoid(z)
        return z * gate, gate + z * gate * torch.sigmoid(-z)
    if act == "gelu_tanh":  # (1 + tanh u) / 2 = sigmoid(2 u)
        u2 = 1.5957691216057308 * z * (1 + 0.044715 * z * z)
        gate = torch.sigmoid(u2)
        return z * gate, gate + z * gate * torch.sigmoid(-u2) * 1.5957691216057308 * (1 + 0.134145 * z * z)
    return z, torch.ones_like(z)


def _d(v):
    return None if v is None else v.double()


def _exact_norm(s):
    k, rms = s["k"], s["rms"]

    def centred(v):
        m = v.sum(1) / k * (0.0 if rms else 1.0)
        return v - m[:, None], m, 1.0 / torch.sqrt((v * v).sum(1) / k - m * m + EPS)

    v = s["b"].double()
    zero = torch.zeros(v.shape[0], dtype=torch.float64, device=v.device)
    m2 = r2 = zero
    if s["post"]:
        c, m2, r2 = centred(v)
        v = c * r2[:, None] * _d(s["pw"])
        if s["pb"] is not None:
            v = v + _d(s["pb"])
    if s["g"] is not None:
        v = torch.mul(v, _d(s["g"]))
    r = torch.add(v, s["x"].double() * (1.0 if s["a"] is None else _d(s["a"])))
    c, m1, r1 = centred(r)
    h = c * r1[:, None] * _d(s["weight"])
    if s["bias"] is not None:
        h = h + _d(s["bias"])
    return r, _round8(h) if s["out"] == "fp8" else h, torch.stack((m1, r1, m2, r2))


def _exact_norm_back(s):
    m1, r1, m2, r2 = s["stats"].double()
    n, centre = s["k"], 0.0 if s["rms"] else 1.0
    dh, w, b = s["dh"].double(), _d(s["weight"]), s["b"].double()
    rh = (s["r"].double() - m1[:, None]) * r1[:, None]

    def through(g, xh, rstd):  # the Jacobian of (x - mean) * rstd, applied from the left
        along = torch.einsum("tc,tc->t", g, xh) / n
        return (g - along[:, None] * xh - centre * (g.sum(1) / n)[:, None]) * rstd[:, None]

    d = through(dh * w, rh, r1) + s["dr"].double()
    a, g, pw, pb = _d(s["a"]), _d(s["g"]), _d(s["pw"]), _d(s["pb"])
    bh = (b - m2[:, None]) * r2[:, None] if s["post"] else b
    s0, s1 = d.sum(0), torch.einsum("tc,tc->c", d, bh)
    one = torch.ones_like(w)
    gate = one if g is None else g
    db = through(d * (gate * pw), bh, r2) if s["post"] else d * gate
    dgate = None if g is None else s1 * (one if pw is None else pw) + (0.0 if pb is None else s0 * pb)
    return (d if a is None else d * a, db, torch.einsum("tc,tc->c", dh, rh), None if s["bias"] is None else dh.sum(0),
            gate * s1 if s["post"] else None, gate * s0 if pb is not None else None, dgate,
            None if a is None else torch.dot(d.flatten(), s["x"].double().flatten()).view(1))


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        return _exact_norm(s)
    if kind == "norm_back":
        return _exact_norm_back(s)
    if kind == "clip":
        norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g.flatten().double())) ** 2 for g in s["grads"]))
        total = torch.tensor(norm, dtype=torch.float64, device="cuda")
        if case["out"] == "none":
            return total
        c = min(1.0, s["max_norm"] / (norm + CLIP_EPS))
        n = 6 * case["layers"]
        big, small = (torch.cat([g.flatten() for g in part]) for part in (s["grads"][:n], s["grads"][n:]))
        return total, big.double() * c, small.double() * c
    if kind == "linear_back":
        dz = s["dy"].double() * _bend(s["z"].double(), case["act"])[1]
        return dz, _round8(dz), dz.sum(0)
    n, k = case["n"], case["k"]
    z = torch.addmm(_d(s["bias"]), _read8(s["x"], 1, k), _read8(s["w"], 128, k).t().contiguous())
    y = _bend(z, case["act"])[0]
    if kind == "mlp":
        y = torch.addmm(_d(s["bias2"]), _round8(y), _read8(s["w2"], 128, n).t().contiguous())
    if s["add"] is not None:
        y = y + s["add"].double()
    return (y, z) if kind == "mlp" else y
