"""residual_norm and its backward pass without a GPU: refusals of the C ABI
(every rejected call returns before any HIP call is made), the binding's checks,
and the oracle's gradients against differences."""
import ctypes

import numpy as np
import pytest
import torch

import muon_newton_schulz_step_amd as mn
from muon_newton_schulz_step_amd import _lib
from oracle import layers_oracle as lo

P = 0x100000  # aligned, never dereferenced by rejected calls
INVALID, UNSUPPORTED, WORKSPACE, OK = (mn.MUON_ERR_INVALID_ARG, mn.MUON_ERR_UNSUPPORTED,
                                       mn.MUON_ERR_WORKSPACE, mn.MUON_OK)
BF16, FP32 = mn.MUON_BF16, mn.MUON_FP32
ALL = dict(weight=P * 20, bias=P * 21, post_weight=P * 22, post_bias=P * 23, gate=P * 24, scale=P * 25)


def t8(k, rows=8, cols=256, block_rows=1, data=None):
    return _lib.MuonTensor8(P * 64 * k if data is None else data, P * 64 * k + P, rows, cols, block_rows)


def params(eps=1e-5, rms=0, **kw):
    return _lib.MuonResidualParams(*[(ALL | kw)[n] for n in ALL], eps, rms)


def forward(x=P, xt=FP32, ldx=256, b=P * 2, bt=BF16, ldb=256, rows=8, cols=256, p=None, r=P * 3,
            ldr=256, h=P * 4, ht=BF16, ldh=256, h8=None, stats=P * 5):
    return mn.lib().muon_residual_norm(x, xt, ldx, b, bt, ldb, rows, cols, p or params(), r, ldr, h,
                                       ht, ldh, h8, stats, None)


BARE = dict(post_weight=0, post_bias=0, gate=0, scale=0)


@pytest.mark.parametrize("kw,expect", [
    (dict(xt=2), INVALID), (dict(bt=3), INVALID), (dict(ht=2), INVALID), (dict(xt=BF16, bt=FP32), UNSUPPORTED),
    (dict(x=0), INVALID), (dict(x=P + 4), INVALID), (dict(ldx=255), INVALID), (dict(ldb=255), INVALID),
    (dict(ldr=255), INVALID), (dict(ldh=255), INVALID), (dict(rows=-1), INVALID), (dict(cols=0), INVALID),
    (dict(b=P * 2 + 2), INVALID), (dict(r=P * 3 + 8), INVALID), (dict(h=P * 4 + 2), INVALID),
    (dict(stats=0), INVALID), (dict(stats=P * 5 + 2), INVALID),
    (dict(p=params(weight=0)), INVALID), (dict(p=params(post_weight=0)), INVALID),
    (dict(p=params(eps=-1.0)), INVALID), (dict(p=params(eps=float("nan"))), INVALID), (dict(p=params(rms=2)), INVALID),
    (dict(p=params(gate=P * 24 + 2)), INVALID),
    (dict(b=0), INVALID),                                          # a gate, but no branch
    (dict(b=0, p=params(post_weight=0, post_bias=0, gate=0), r=0), INVALID),  # scaled, but not written
    (dict(r=0), INVALID), (dict(h=0), INVALID), (dict(h8=t8(1)), INVALID),
    (dict(h=0, h8=t8(1, 8, 255)), INVALID), (dict(h=0, h8=t8(1, 8, 256, 128)), INVALID),
    (dict(h=0, h8=t8(1, data=P)), INVALID), (dict(r=P), INVALID), (dict(r=P * 2), INVALID),
    (dict(h=P * 3), INVALID), (dict(stats=P * 3), INVALID), (dict(stats=P * 20), INVALID), (dict(r=P * 25), INVALID),
    (dict(cols=16385, ldx=16385, ldb=16385, ldr=16385, ldh=16385), UNSUPPORTED),
    (dict(rows=0), OK), (dict(rows=0, x=0, b=0, r=0, h=0, stats=0), OK),
    (dict(rows=0, h=0, h8=t8(1, 0)), OK),
])
def test_forward_refusals(kw, expect):
    if expect == UNSUPPORTED and "cols" in kw:  # large rows that do not meet
        kw = kw | dict(rows=1)
    assert forward(**kw) == expect


def backward(dr=P, dh=P * 2, r=P * 3, b=P * 4, x=P * 5, xt=FP32, bt=BF16, rows=8, cols=256, p=None,
             stats=P * 6, dx=P * 7, db=P * 8, g=None, accumulate=0, ws=P * 9, ws_bytes=1 << 20, ld=None):
    ld = ld or {}
    names = ("weight", "bias", "post_weight", "post_bias", "gate", "scale")
    grads = _lib.MuonResidualGrads(*[({n: P * (30 + i) for i, n in enumerate(names)} | (g or {}))[n] for n in names])
    return mn.lib().muon_residual_norm_backward(
        dr, ld.get("dr", cols), dh, ld.get("dh", cols), r, ld.get("r", cols), b, ld.get("b", cols), x,
        ld.get("x", cols), xt, bt, rows, cols, p or params(), stats, dx, ld.get("dx", cols), db,
        ld.get("db", cols), ctypes.byref(grads), accumulate, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(xt=2), INVALID), (dict(bt=2), INVALID), (dict(xt=BF16, bt=FP32), UNSUPPORTED),
    (dict(accumulate=2), INVALID), (dict(dh=0), INVALID), (dict(r=0), INVALID), (dict(dx=0), INVALID),
    (dict(b=0), INVALID), (dict(x=0), INVALID), (dict(dr=P + 2), INVALID), (dict(db=P * 8 + 2), INVALID),
    (dict(stats=0), INVALID), (dict(p=params(weight=0)), INVALID), (dict(g=dict(gate=P * 34 + 2)), INVALID),
    *[(dict(ld={n: 255}), INVALID) for n in ("dr", "dh", "r", "b", "x", "dx", "db")],
    (dict(p=params(gate=0)), INVALID), (dict(p=params(scale=0)), INVALID),  # gradients of what is not there
    (dict(p=params(post_bias=0)), INVALID),
    (dict(p=params(post_weight=0, post_bias=0)), INVALID),
    (dict(ws=0), WORKSPACE), (dict(ws=P * 9 + 16), WORKSPACE), (dict(ws_bytes=4351), WORKSPACE),
    (dict(ws=P), INVALID), (dict(dx=P), INVALID), (dict(dx=P * 5), INVALID), (dict(db=P * 7), INVALID),
    (dict(g=dict(weight=P * 20)), INVALID), (dict(g=dict(weight=P * 31)), INVALID), (dict(g=dict(scale=P * 6)), INVALID),
    (dict(cols=16385, rows=1), UNSUPPORTED),
    (dict(rows=0, accumulate=1), OK), (dict(rows=0, accumulate=1, dr=0, dh=0, r=0, b=0, x=0, dx=0, db=0, stats=0, ws=0), OK),
])
def test_backward_refusals(kw, expect):
    assert backward(**kw) == expect


def test_workspace_sizes():
    f = mn.residual_norm_backward_workspace_bytes
    assert f(8, 256, True) == 256 + 4 * 256 * 4 and f(8, 256, False) == 256 + 2 * 256 * 4
    assert f(10 ** 6, 4096, True) == 2048 + 256 * 4 * 4096 * 4
    assert f(0, 8, True) == f(8, 0, True) == f(8, 16385, True) == f(1 << 40, 8, True) == 0


def test_binding_refusals():
    x, w = torch.zeros(4, 8), torch.ones(8)
    for kw in (dict(), dict(post_bias=w), dict(gate=torch.ones(7)), dict(scale=torch.tensor(1.0)),
               dict(gate=w.double()), dict(branch=torch.zeros(4, 7)), dict(branch=None, gate=w)):
        kw = dict(branch=x) | kw
        with pytest.raises(ValueError):        # (the first: not on a GPU)
            mn.residual_norm(x, kw.pop("branch"), w, **kw)
    st = torch.zeros(4, 4)
    for kw in (dict(), dict(stats=st[:2]), dict(dr=x.double()), dict(dh=torch.zeros(4, 7)), dict(gate=w, branch=None),
               dict(scale=torch.ones(1)), dict(accumulate=True), dict(branch=x.bfloat16())):
        a = dict(dr=x, dh=x, r=x, branch=x, weight=w, stats=st) | kw
        with pytest.raises(ValueError):
            mn.residual_norm_backward(a.pop("dr"), a.pop("dh"), a.pop("r"), a.pop("branch"),
                                      a.pop("weight"), a.pop("stats"), **a)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("post,gate,scale", [(1, 1, 1), (0, 1, 0), (1, 0, 0), (0, 0, 1), (0, 0, 0)])
def test_oracle_gradients(rms, post, gate, scale):
    rng = np.random.default_rng(3)
    rows, n = 3, 7
    v = dict(x=rng.normal(size=(rows, n)), branch=rng.normal(size=(rows, n)) + 0.5, w=rng.normal(size=n),
             b=rng.normal(size=n), pw=rng.normal(size=n) if post else None,
             pb=rng.normal(size=n) if post else None, gate=rng.normal(size=n) if gate else None,
             scale=np.array([0.7]) if scale else None)
    gr, gh = rng.normal(size=(rows, n)), rng.normal(size=(rows, n))

    def loss(**kw):
        r, h, _ = lo.residual_norm(**(v | kw), rms=rms)
        return float((r * gr).sum() + (h * gh).sum())

    r, _, stats = lo.residual_norm(**v, rms=rms)
    got = lo.residual_norm_backward(gr, gh, r, v["branch"], v["w"], stats, v["x"], v["pw"], v["pb"],
                                    v["gate"], v["scale"], rms)
    names = dict(dx="x", dbranch="branch", dweight="w", dbias="b", dpost_weight="pw", dpost_bias="pb",
                 dgate="gate", dscale="scale")
    for name, of in names.items():
        if v[of] is None:
            continue
        num = np.zeros(v[of].size)
        for i in range(v[of].size):
            e = np.zeros(v[of].size)
            e[i] = 1e-6
            e = e.reshape(v[of].shape)
            num[i] = (loss(**{of: v[of] + e}) - loss(**{of: v[of] - e})) / 2e-6
        assert np.max(np.abs(num - np.asarray(got[name]).reshape(-1))) < 1e-7, name
