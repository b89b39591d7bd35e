"""residual_norm and its backward pass on the GPU against the 64-bit oracle.

Bounds.  u = 2^-24.  A lane adds at most 24 numbers of a row one after the other,
a wave its 64 lanes in 6 steps and a team its 16 waves one by one: a row's sum is
off by at most D = 48 u times the sum of magnitudes.  With inputs that are off by e:
  mean     dm = mean(e) + D mean|v| + u |mean|
  variance 2 mean|c| (dm + e) + 3 (dm + max e)^2 + (D + 4 u) var,  c = v - mean
  rstd     relative half of that over var + eps, + 4 u
  vh       rstd (dm + e + u |c|) + |vh| (that + u)
and each product and sum after it adds u of its own.  The backward pass's
formulas are bounded the same way, term by term; a column's sum of `rows` terms is
off by at most rows u of their magnitudes.  Results in bf16 add 2^-8 of the value,
those in 8 bits 2^-4, or 2^-10 of the block's scale."""
import numpy as np
import pytest
import torch

import muon_newton_schulz_step_amd as mn
from gpu_helpers import announce, to64
from oracle import layers_oracle as lo

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24
HALF = {BF16: 2.0 ** -8, FP32: U}
D = 48 * U
EPS = 1e-5
TYPES = [(BF16, BF16), (FP32, BF16), (FP32, FP32)]


def randn(*shape, seed=0, std=1.0, mean=0.0, dtype=FP32):
    g = torch.Generator(DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * std + mean).to(dtype)


def make(rows, cols, xt, bt, rms, post, gate, scale, bias, seed=0):
    x = (randn(rows, cols, seed=seed) * torch.exp(randn(rows, 1, seed=seed + 1)) + 0.3).to(xt)
    return dict(x=x, branch=randn(rows, cols, seed=seed + 2, std=2.0, mean=0.2, dtype=bt),
                weight=randn(cols, seed=seed + 3, std=0.2, mean=1.0),
                bias=randn(cols, seed=seed + 4, std=0.2) if bias else None,
                post_weight=randn(cols, seed=seed + 5, std=0.2, mean=1.0) if post else None,
                post_bias=randn(cols, seed=seed + 6, std=0.2) if post and bias else None,
                gate=randn(cols, seed=seed + 7, std=0.3, mean=0.5) if gate else None,
                scale=randn(1, seed=seed + 8, std=0.1, mean=0.9) if scale else None, rms=rms)


def opt64(v):
    return None if v is None else to64(v)


def oracle_args(a):
    return dict(w=to64(a["weight"]), b=opt64(a["bias"]), pw=opt64(a["post_weight"]),
                pb=opt64(a["post_bias"]), gate=opt64(a["gate"]), scale=opt64(a["scale"]), rms=a["rms"])


def mag(v, otherwise=1.0):
    return otherwise if v is None else np.abs(v)


def norm_bound(v, e, rms, eps):
    """(vh, its bound, mean's, rstd's) of a norm of v, off by e."""
    vh, mean, rstd = lo._norm(v, rms, eps)
    c, var = v - mean[:, None], 1 / rstd ** 2 - eps
    av = np.abs(v).mean(1)
    dm = np.zeros_like(mean) if rms else e.mean(1) + D * av + U * np.abs(mean)
    dvar = 2 * (np.abs(c) * (dm[:, None] + e)).mean(1) + 3 * (dm + e.max(1)) ** 2 + (D + 4 * U) * var
    rel = 0.5 * dvar * rstd ** 2 * (1 + dvar * rstd ** 2) + 4 * U
    bound = rstd[:, None] * (dm[:, None] + e + U * np.abs(c)) + np.abs(vh) * (rel[:, None] + U)
    return vh, bound, dm, rel * rstd


def inside(got, ref, bound, what):
    got = to64(got.float()) if torch.is_tensor(got) else got
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           float(np.nanmax(np.abs(got - ref) / np.maximum(bound, 1e-300))))


def values8(t):
    q = to64(t.data.float())[:, :t.cols]
    scale = lo.expand(t.scale.cpu().numpy().astype(np.int64)[:, :-(-t.cols // 128)] - 127, q.shape, 1)
    return q * scale, scale


def check_forward(a, out, eps=EPS):
    r, h, stats = mn.residual_norm(a["x"], a["branch"], a["weight"], a["bias"], post_weight=a["post_weight"],
                                   post_bias=a["post_bias"], gate=a["gate"], scale=a["scale"],
                                   rms=a["rms"], eps=eps, out_dtype=out)
    o, x = oracle_args(a), to64(a["x"])
    rref, href, sref = lo.residual_norm(x, opt64(a["branch"]), **o, eps=eps)
    assert r.dtype == a["x"].dtype and stats.shape == (4, x.shape[0])
    er = U * np.abs(x) * mag(o["scale"])
    if a["branch"] is not None:
        p = to64(a["branch"])
        ep = np.zeros_like(p)
        if o["pw"] is not None:
            ph, eph, dm, ds = norm_bound(p, ep, a["rms"], eps)
            inside(stats[2], sref[2], dm, "post mean")
            inside(stats[3], sref[3], ds, "post rstd")
            p = ph * o["pw"]
            ep = eph * np.abs(o["pw"]) + 3 * U * np.abs(p)
            p = np.abs(p) + mag(o["pb"], 0.0)
        er = er + mag(o["gate"]) * (ep + 3 * U * np.abs(p))
    if a["branch"] is None or o["pw"] is None:
        assert (stats[2:] == 0).all()
    er = er + U * np.abs(rref)
    inside(r, rref, er + HALF[r.dtype] * (np.abs(rref) + er), "r")
    rh, erh, dm, ds = norm_bound(rref, er, a["rms"], eps)
    inside(stats[0], sref[0], dm, "mean")
    inside(stats[1], sref[1], ds, "rstd")
    eh = erh * np.abs(o["w"]) + 3 * U * (np.abs(rh * o["w"]) + mag(o["b"], 0.0))
    if out == E4M3:
        hv, scale = values8(h)
        n = x.shape[1]
        blocks = lambda v: np.pad(v, ((0, 0), (0, -n % 128))).reshape(len(v), -1, 128).max(2)  # noqa: E731
        s = scale[:, ::128]
        assert (blocks(np.abs(href) - eh) <= 448 * s).all()
        assert ((blocks(np.abs(href) + eh) >= 224 * s) | (s <= 2.0 ** -117)).all()
        inside(hv, href, eh + np.maximum(2.0 ** -4 * (np.abs(href) + eh), 2.0 ** -10 * scale), "h")
        assert torch.count_nonzero(h.data.view(torch.uint8)[:, n:]) == 0
        assert (h.scale[:, -(-n // 128):] == 10).all()
    else:
        assert h.dtype == out
        inside(h, href, eh + HALF[out] * (np.abs(href) + eh), "h")
    return r, h, stats


def check_backward(a, r, stats, dr_there=True, seed=50, **kw):
    rows, cols = a["x"].shape
    bt = (a["x"] if a["branch"] is None else a["branch"]).dtype
    dr = randn(rows, cols, seed=seed, dtype=a["x"].dtype) if dr_there else None
    dh = randn(rows, cols, seed=seed + 1, dtype=bt)
    got = mn.residual_norm_backward(dr, dh, r, a["branch"], a["weight"], stats, x=a["x"],
                                    bias=a["bias"] is not None, post_weight=a["post_weight"],
                                    post_bias=a["post_bias"], gate=a["gate"], scale=a["scale"],
                                    rms=a["rms"], **kw)
    o = oracle_args(a)
    o.pop("b")
    w = o.pop("w")
    ref = lo.residual_norm_backward(opt64(dr), to64(dh), to64(r), opt64(a["branch"]), w, to64(stats),
                                    to64(a["x"]), **o)
    st = to64(stats)[:, :, None]
    rd, h = np.abs(opt64(dr)) if dr_there else 0.0, to64(dh)
    rh = (to64(r) - st[0]) * st[1]
    g = h * w
    mean = lambda v: np.abs(v).mean(1, keepdims=True)  # noqa: E731
    c0, c1 = 0.0 if a["rms"] else g.mean(1, keepdims=True), (g * rh).mean(1, keepdims=True)
    e = st[1] * ((D + 4 * U) * mean(g) + np.abs(rh) * (D + 8 * U) * mean(g * rh)
                 + 8 * U * (np.abs(g) + np.abs(c0) + np.abs(rh * c1))) + 2 * U * rd
    d = ref["dx"] / _or1(o["scale"])
    e = e + 2 * U * np.abs(d)
    lim = lambda v, ev, dt: ev + HALF[dt] * (np.abs(v) + ev)  # noqa: E731
    s = mag(o["scale"])
    inside(got.dx, ref["dx"], lim(ref["dx"], s * e + U * np.abs(ref["dx"]), got.dx.dtype), "dx")
    col = lambda terms, et: et.sum(0) + rows * U * (np.abs(terms) + et).sum(0)  # noqa: E731
    inside(got.dweight, ref["dweight"], col(h * rh, 4 * U * np.abs(h * rh)), "dweight")
    if a["bias"] is None:
        assert got.dbias is None
    else:
        inside(got.dbias, ref["dbias"], col(h, 0 * h), "dbias")
    if o["scale"] is None:
        assert got.dscale is None
    else:
        x = np.abs(to64(a["x"]))
        inside(got.dscale, np.array([ref["dscale"]]), (e * x + 28 * U * np.abs(d) * x).sum() + U * abs(ref["dscale"]), "dscale")
    if a["branch"] is None:
        assert got[1] is None and got[4:7] == (None, None, None)
        return got, ref
    b = to64(a["branch"])
    bh = (b - st[2]) * st[3] if o["pw"] is not None else b
    gate, pw = mag(o["gate"]), mag(o["pw"])
    ee = gate * pw * (e + 2 * U * np.abs(d))
    ev = gate * pw * np.abs(d)
    if o["pw"] is None:
        eb = ee
        assert got.dpost_weight is None and got.dpost_bias is None
    else:
        m = lambda v: v.mean(1, keepdims=True)  # noqa: E731
        e0 = 0.0 if a["rms"] else m(ee) + (D + 4 * U) * m(ev)
        e1 = m(ee * np.abs(bh)) + (D + 8 * U) * m(ev * np.abs(bh))
        eb = st[3] * (ee + e0 + np.abs(bh) * e1 + 8 * U * (ev + (0 if a["rms"] else m(ev)) + np.abs(bh) * m(ev * np.abs(bh))))
        eb = eb + 2 * U * np.abs(ref["dbranch"])
        gs = gate if np.ndim(gate) else np.ones(cols)
        inside(got.dpost_weight, ref["dpost_weight"], gs * col(d * bh, (e + 4 * U * np.abs(d)) * np.abs(bh)) + U * np.abs(ref["dpost_weight"]), "dpost_weight")
        if o["pb"] is None:
            assert got.dpost_bias is None
        else:
            inside(got.dpost_bias, ref["dpost_bias"], gs * col(d, e) + U * np.abs(ref["dpost_bias"]), "dpost_bias")
    inside(got.dbranch, ref["dbranch"], lim(ref["dbranch"], eb, got.dbranch.dtype), "dbranch")
    if o["gate"] is None:
        assert got.dgate is None
    else:
        b1, b0 = col(d * bh, (e + 4 * U * np.abs(d)) * np.abs(bh)), col(d, e)
        tot = pw * (np.abs((d * bh).sum(0)) + b1) + mag(o["pb"], 0.0) * (np.abs(d.sum(0)) + b0)
        inside(got.dgate, ref["dgate"], pw * b1 + mag(o["pb"], 0.0) * b0 + 2 * U * tot, "dgate")
    return got, ref


def _or1(v):
    return 1.0 if v is None else v


SIZES = [(1, 1), (2, 7), (3, 128), (1, 512), (5, 513), (33, 1000), (2, 1027), (9, 1280), (3, 1536), (4, 1540),
         (17, 2047), (6, 4096), (3, 2500), (2, 5000), (3, 8192), (2, 8200), (3, 16384), (700, 200), (1100, 600),
         (2100, 1100), (530, 2050)]


@pytest.mark.parametrize("xt,bt", TYPES)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_all_options(rows, cols, xt, bt):
    """Every combination of two of the options in turn over the sizes, forward and backward."""
    k = SIZES.index((rows, cols)) + TYPES.index((xt, bt))
    outs = (BF16, FP32, E4M3)
    for j, (post, gate, scale, rms, bias) in enumerate((
            (1, 1, 1, k % 2, 1), (0, 0, 0, (k + 1) % 2, k % 2), (1, 0, 0, k % 2, 0),
            (0, 1, 1, (k + 1) % 2, 1), (1, 1, 0, (k + 1) % 2, 1), (0, 0, 1, k % 2, 0))):
        announce("residual_norm", rows, cols, xt, bt, "post", post, "gate", gate, "scale", scale, "rms", rms)
        a = make(rows, cols, xt, bt, bool(rms), post, gate, scale, bias, seed=100 * j)
        r, _, stats = check_forward(a, outs[(j + k) % 3])
        check_backward(a, r, stats, dr_there=(j + k) % 4 != 0)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("out", [BF16, FP32, E4M3])
@pytest.mark.parametrize("xt", [BF16, FP32])
def test_without_branch(xt, out, rms):
    for scale in (0, 1):
        for rows, cols in ((1, 768), (40, 1280), (3, 4100)):
            announce("residual_norm without a branch", xt, out, rms, scale, rows, cols)
            a = make(rows, cols, xt, xt, rms, 0, 0, scale, not rms, seed=9)
            a["branch"] = None
            r, _, stats = check_forward(a, out)
            assert (r is a["x"]) == (not scale)
            check_backward(a, r, stats)
            check_backward(a, r, stats, dr_there=False)


def test_as_layer_norm():
    """Without a branch it is layer_norm, to rounding."""
    announce("residual_norm as layer_norm")
    x, w, b = randn(50, 1280, seed=1), randn(1280, seed=2), randn(1280, seed=3)
    _, h, stats = mn.residual_norm(x, None, w, b)
    y, mean, rstd = mn.layer_norm(x, w, b)
    assert torch.allclose(h, y, rtol=1e-5, atol=1e-5)
    assert torch.allclose(stats[0], mean, rtol=1e-5, atol=1e-6) and torch.allclose(stats[1], rstd, rtol=1e-5)


def test_same_gradient_is_one_tensor():
    announce("residual_norm: dx and dbranch")
    a = make(20, 300, BF16, BF16, True, 0, 0, 0, 0)
    r, _, stats = check_forward(a, BF16)
    got, _ = check_backward(a, r, stats)
    assert got.dbranch is got.dx
    a = make(20, 300, FP32, BF16, True, 0, 0, 0, 0)
    r, _, stats = check_forward(a, BF16)
    got, _ = check_backward(a, r, stats)
    assert torch.equal(got.dbranch, got.dx.to(BF16))


def test_flat_rows_and_large_means():
    """Rows of equal values, of little variance around a large mean, of zeros."""
    announce("residual_norm: flat rows")
    for xt, bt in TYPES:
        rows, cols = 6, 1280
        x = torch.zeros(rows, cols, device=DEV)
        x[1], x[2], x[3] = 1000.0, 3.0, -0.5
        x[4] = 1000.0 + randn(cols, seed=3, std=0.01)
        b = torch.zeros(rows, cols, device=DEV)
        b[1], b[2], b[5] = 7.0, -3.0, 512.0
        a = make(rows, cols, xt, bt, False, 0, 0, 0, 1)
        a["x"], a["branch"] = x.to(xt), b.to(bt)
        r, h, stats = mn.residual_norm(a["x"], a["branch"], a["weight"], a["bias"], out_dtype=FP32)
        flat = [0, 1, 2, 3, 5]
        # r is exact, all its deviations are zero and h is the bias
        assert torch.equal(h[flat], a["bias"].expand(5, -1)) and torch.equal(r[flat], (x + b)[flat].to(xt))
        assert torch.equal(stats[0][flat], (x + b)[flat, 0])
        r, _, stats = mn.residual_norm(a["x"], a["branch"], a["weight"], a["bias"], rms=True, out_dtype=FP32)
        assert (stats[0] == 0).all() and torch.isfinite(stats).all()


def test_not_finite():
    announce("residual_norm: not finite")
    for out in (BF16, FP32, E4M3):
        a = make(9, 700, FP32, BF16, False, 1, 1, 1, 1)
        kw = dict(post_weight=a["post_weight"], post_bias=a["post_bias"], gate=a["gate"], scale=a["scale"], out_dtype=out)
        plain = lambda h: h.dequantize(FP32) if out == E4M3 else h.float()  # noqa: E731
        ref = mn.residual_norm(a["x"], a["branch"], a["weight"], a["bias"], **kw)
        a["x"][2, 5], a["branch"][4, 600], a["x"][6, 0] = float("inf"), float("nan"), float("nan")
        r, h, stats = mn.residual_norm(a["x"], a["branch"], a["weight"], a["bias"], **kw)
        good = [0, 1, 3, 5, 7, 8]
        assert torch.equal(r[good], ref[0][good]) and torch.equal(plain(h)[good], plain(ref[1])[good])
        assert torch.equal(stats[:, good], ref[2][:, good])
        for row in (2, 4, 6):
            assert torch.isnan(plain(h)[row]).any()
        assert torch.isinf(r[2, 5]) and torch.isnan(r[4]).all() and torch.isnan(r[6, 0])


def test_strides_and_what_lies_around():
    announce("residual_norm: strides")
    rows, cols = 37, 520
    a = make(rows, cols, FP32, BF16, False, 1, 1, 1, 1)
    ref = mn.residual_norm(a["x"], a["branch"], a["weight"], a["bias"], post_weight=a["post_weight"], post_bias=a["post_bias"],
                           gate=a["gate"], scale=a["scale"])
    wide = {n: torch.zeros(rows, cols + 24, dtype=a[n].dtype, device=DEV) for n in ("x", "branch")}
    for n, t in wide.items():
        t[:, 8:8 + cols] = a[n]
    got = mn.residual_norm(wide["x"][:, 8:8 + cols], wide["branch"][:, 8:8 + cols], a["weight"], a["bias"],
                           post_weight=a["post_weight"], post_bias=a["post_bias"], gate=a["gate"], scale=a["scale"])
    assert all(torch.equal(p, q) for p, q in zip(ref, got))
    dr, dh = randn(rows, cols + 8, seed=1)[:, :cols], randn(rows, cols + 8, seed=2, dtype=BF16)[:, :cols]
    kw = dict(post_weight=a["post_weight"], post_bias=a["post_bias"], gate=a["gate"], scale=a["scale"])
    one = mn.residual_norm_backward(dr, dh, got[0], wide["branch"][:, 8:8 + cols], a["weight"], got[2],
                                    x=wide["x"][:, 8:8 + cols], **kw)
    two = mn.residual_norm_backward(dr.contiguous(), dh.contiguous(), ref[0], a["branch"], a["weight"], ref[2], x=a["x"], **kw)
    assert all(torch.equal(p, q) for p, q in zip(one, two))


def test_into_and_accumulate():
    announce("residual_norm: accumulation")
    a = make(300, 640, FP32, BF16, False, 1, 1, 1, 1)
    r, _, stats = check_forward(a, BF16)
    got, _ = check_backward(a, r, stats)
    into = mn.ResidualNormGrads(None, None, *[torch.full_like(g, 2.0) for g in got[2:]])
    dr, dh = randn(300, 640, seed=50), randn(300, 640, seed=51, dtype=BF16)
    kw = dict(x=a["x"], post_weight=a["post_weight"], post_bias=a["post_bias"], gate=a["gate"], scale=a["scale"])
    again = mn.residual_norm_backward(dr, dh, r, a["branch"], a["weight"], stats, into=into, accumulate=True, **kw)
    for p, q, g in zip(again[2:], into[2:], got[2:]):
        assert p is q and torch.equal(p, g + 2.0)
    again = mn.residual_norm_backward(dr, dh, r, a["branch"], a["weight"], stats, into=into, **kw)
    assert all(torch.equal(p, g) for p, g in zip(again[2:], got[2:]))
    empty = mn.residual_norm_backward(dr[:0], dh[:0], r[:0], a["branch"][:0], a["weight"], stats[:, :0].contiguous(),
                                      into=into, accumulate=True, **(kw | dict(x=a["x"][:0])))
    assert all(torch.equal(p, g) for p, g in zip(empty[2:], got[2:]))
    empty = mn.residual_norm_backward(dr[:0], dh[:0], r[:0], a["branch"][:0], a["weight"], stats[:, :0].contiguous(),
                                      **(kw | dict(x=a["x"][:0])))
    assert all((g == 0).all() for g in empty[2:]) and empty.dx.shape == (0, 640)
    with pytest.raises(ValueError):
        mn.residual_norm_backward(dr, dh, r, a["branch"], a["weight"], stats, into=into, **(kw | dict(gate=None)))
    with pytest.raises(mn.MuonError):
        mn.residual_norm_backward(dr, dh, r, a["branch"], a["weight"], stats, workspace=torch.empty(64, dtype=torch.uint8, device=DEV), **kw)


def test_repeats_graph_and_stream():
    announce("residual_norm captured, on another stream")
    a = make(700, 1280, FP32, BF16, False, 1, 1, 1, 1)
    dr, dh = randn(700, 1280, seed=1), randn(700, 1280, seed=2, dtype=BF16)
    kw = dict(post_weight=a["post_weight"], post_bias=a["post_bias"], gate=a["gate"], scale=a["scale"])

    def both():
        r, h, stats = mn.residual_norm(a["x"], a["branch"], a["weight"], a["bias"], out_dtype=E4M3, **kw)
        back = mn.residual_norm_backward(dr, dh, r, a["branch"], a["weight"], stats, x=a["x"], **kw)
        return [r, h.data.view(torch.uint8), h.scale, stats, *back]

    ref = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = both()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(ref, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for seed in (7, 8, 9):
        a["x"].copy_(randn(700, 1280, seed=seed))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        eager = both()
        assert all(torch.equal(p, q) for p, q in zip(kept, eager))
