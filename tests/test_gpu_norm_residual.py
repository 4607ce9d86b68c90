"""switch_layer_norm_residual and its backward pass against the formulas in 64 bits.

Tolerances.  Forward: every value is a sum of a few products of rounded fp32
numbers: at most 16 roundings (u = 2^-24 each) of terms no larger than their
absolute sum, a row sum over d columns adding at most (d / 256 + 12) u
(the running sum of a thread, five shuffles, up to 16 warps, in a mean whose
error enters by half or once), and half a step of the output type.  Backward: the
same on sums of absolute terms; a column sum over T rows adds a running sum of at
most T / 2 + 300 rows in sequence, u each.
"""
from __future__ import annotations

import pytest
import torch

import sparse_mixture_experts_argmax_b200 as swl
from sparse_mixture_experts_argmax_b200 import build as swl_build

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    swl_build.build()
    swl.lib()


def _hat(v, kind):
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    return v / (v.square().mean(1, keepdim=True) + EPS).sqrt()


def _affine(v, w, b, kind):
    o = _hat(v, kind) * w
    return o if b is None else o + b


def _branch(a, kind):
    u = a["y"] if a.get("w_post") is None else _affine(a["y"], a["w_post"], a.get("b_post"), kind)
    if a.get("scale") is not None:
        u = u * a["scale"]
    return u if a.get("gate") is None else u * a["gate"][:, None]


def _inputs(T, d, dtype, kind, post, pre, gate, scale, bias, y=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    a = {"x": (n(T, d) + 0.3).to(dtype)}
    if y:
        a["y"] = (n(T, d) * 0.7 - 0.2).to(dtype)
        a["y"][::7] = 0                              # dropped tokens
        if gate:
            a["gate"] = torch.rand(T, generator=g, device="cuda")
            a["gate"][::7] = 0
        if scale:
            a["scale"] = 0.3 + 0.1 * n(d)
        if post:
            a["w_post"] = 1 + 0.2 * n(d)
            if bias and kind == "layer":
                a["b_post"] = 0.2 * n(d)
    if pre:
        a["w_pre"] = 1 + 0.2 * n(d)
        if bias and kind == "layer":
            a["b_pre"] = 0.2 * n(d)
    return a


def _row_u(d):
    return (d / 256 + 12) * U


def _check_forward(a, out, kind, T, d):
    dt = a["x"].dtype
    D = {k: v.double() for k, v in a.items()}
    r = D["x"] + _branch(D, kind) if "y" in a else D["x"]
    if "y" in a:
        size = D["x"].abs() + _branch(D, kind).abs()
        if a.get("w_post") is not None:             # hat and bias may cancel; the mean's own size
            mean = D["y"].abs().mean(1, keepdim=True)
            spread = (D["y"].var(1, unbiased=False, keepdim=True) + EPS).sqrt()
            part = (_hat(D["y"], kind).abs() + mean / spread) * a["w_post"].abs().double()
            if a.get("b_post") is not None:
                part = part + a["b_post"].abs().double()
            for k in ("scale",):
                part = part * a[k].abs().double() if a.get(k) is not None else part
            size = size + (part * a["gate"].double()[:, None] if a.get("gate") is not None else part)
        tol = size * (16 * U + 2 * _row_u(d)) + HALF[dt] * r.abs() + 1e-30
        assert ((out["r"].double() - r).abs() <= tol).all()
    else:
        assert out["r"] is a["x"]
        size = D["x"].abs()
    if a.get("w_pre") is None:
        assert out["h"] is None
        return
    h = _affine(r, D["w_pre"], D.get("b_pre"), kind)
    std = ((r - r.mean(1, keepdim=True)) if kind == "layer" else r).square().mean(1, keepdim=True)
    rho = 1 / (std + EPS).sqrt()
    # r's own error is amplified by rho w (and, through the statistics, by |r^|)
    er = size * (16 * U + 2 * _row_u(d))
    worst = er.square().mean(1, keepdim=True).sqrt() + er
    tol = 3 * rho * worst * D["w_pre"].abs() * (1 + _hat(r, kind).abs())
    tol = tol + (h.abs() + (r.abs() + r.abs().mean(1, keepdim=True)) * rho * D["w_pre"].abs()) * (
        16 * U + 2 * _row_u(d)) + HALF[dt] * h.abs() + 1e-30
    assert ((out["h"].double() - h).abs() <= tol).all()


CASES = [(1, 8), (3, 1), (5, 37), (130, 64), (33, 256), (17, 257), (9, 300), (129, 768), (64, 771),
         (40, 1000), (33, 1026), (300, 2048), (65, 4096), (6, 5000), (11, 8192), (4, 8190), (3, 16384),
         (2, 9001)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,d", CASES)
def test_forward(T, d, kind, dtype):
    for seed, flags in enumerate([(1, 1, 1, 1, 1), (0, 1, 1, 0, 0), (1, 0, 0, 1, 1), (0, 0, 0, 0, 0),
                                  (1, 1, 0, 0, 0)]):
        post, pre, gate, scale, bias = flags
        a = _inputs(T, d, dtype, kind, post, pre, gate, scale, bias, seed=seed)
        out = swl.norm_residual(kind=kind, eps=EPS, **a)
        _check_forward(a, out, kind, T, d)
    a = _inputs(T, d, dtype, kind, 0, 1, 0, 0, 1, y=False)
    _check_forward(a, swl.norm_residual(kind=kind, eps=EPS, **a), kind, T, d)


def _grads64(a, dr, dh, r_saved, kind):
    """(gradients, sums of the absolute terms of the column sums) in 64 bits.  r is
    the saved (rounded) residual, a constant plus the branch."""
    D = {k: v.double() for k, v in a.items()}
    leaf = {k: v.clone().requires_grad_() for k, v in D.items()}
    if "y" in a:
        x0 = (r_saved.double() - _branch(D, kind)).requires_grad_()
        r = x0 + _branch(leaf, kind)
    else:
        x0 = r_saved.double().requires_grad_()
        r = x0
    total = (r * 0).sum() if dr is None else (dr.double() * r).sum()
    if dh is not None:
        total = total + (dh.double() * _affine(r, leaf["w_pre"], leaf.get("b_pre"), kind)).sum()
    names = [k for k in a if k != "x"]
    got = torch.autograd.grad(total, [x0] + [leaf[k] for k in names])
    return {"d" + k: v for k, v in zip(["x"] + names, got)}


def _check_backward(a, kind, T, d, use_dr, seed):
    dt = a["x"].dtype
    g = torch.Generator(device="cuda").manual_seed(100 + seed)
    r = swl.norm_residual(kind=kind, eps=EPS, **a)["r"]
    dr = (torch.randn((T, d), generator=g, device="cuda") * 0.1).to(dt) if use_dr else None
    dh = None
    if a.get("w_pre") is not None:
        dh = (torch.randn((T, d), generator=g, device="cuda") * 0.1).to(dt)
    args = {k: v for k, v in a.items() if k != "x"}
    got = swl.norm_residual_backward(dr, dh, r, kind=kind, eps=EPS, **args)
    want = _grads64(a, dr, dh, r, kind)
    D = {k: v.double() for k, v in a.items()}
    rd = r.double()
    # sizes of the terms: rows of D, its row means, and what the norms multiply them by
    size = torch.zeros_like(rd) if dr is None else dr.double().abs()
    hat_r = None
    if dh is not None:
        rho = 1 / ((rd - rd.mean(1, keepdim=True) if kind == "layer" else rd).square().mean(
            1, keepdim=True) + EPS).sqrt()
        hat_r = _hat(rd, kind).abs() + rd.abs().mean(1, keepdim=True) * rho
        t = dh.double().abs() * D["w_pre"].abs()
        size = size + rho * (t + t.mean(1, keepdim=True) + hat_r * (t * hat_r).mean(1, keepdim=True))
    rel = 24 * U + 4 * _row_u(d)
    tiny = 1e-30

    def ok(name, tol):
        diff = (got[name].double() - want[name]).abs()
        assert (diff <= tol + tiny).all(), (name, float((diff / (tol + tiny)).max()))

    ok("dx", size * rel + HALF[dt] * want["dx"].abs())
    rows = (T / 2 + 300) * U + rel
    if dh is not None:
        ok("dw_pre", (dh.double().abs() * hat_r).sum(0) * rows)
        if a.get("b_pre") is not None:
            ok("db_pre", dh.double().abs().sum(0) * rows)
    if "y" not in a:
        assert got["dy"] is None and got["dgate"] is None
        return
    gate = D["gate"][:, None] if a.get("gate") is not None else torch.ones_like(rd[:, :1])
    scale = D["scale"].abs() if a.get("scale") is not None else 1.0
    u = D["y"].abs()
    du = size * gate * scale
    dy = du
    if a.get("w_post") is not None:
        y = D["y"]
        rho = 1 / ((y - y.mean(1, keepdim=True) if kind == "layer" else y).square().mean(
            1, keepdim=True) + EPS).sqrt()
        hat = _hat(y, kind).abs() + y.abs().mean(1, keepdim=True) * rho
        u = hat * D["w_post"].abs() + (D["b_post"].abs() if a.get("b_post") is not None else 0.0)
        t = du * D["w_post"].abs()
        dy = rho * (t + t.mean(1, keepdim=True) + hat * (t * hat).mean(1, keepdim=True))
        ok("dw_post", (du * hat).sum(0) * rows)
        if a.get("b_post") is not None:
            ok("db_post", du.sum(0) * rows)
    ok("dy", dy * rel + HALF[dt] * want["dy"].abs())
    if a.get("gate") is not None:
        ok("dgate", (size * scale * u).sum(1) * rel)
    if a.get("scale") is not None:
        ok("dscale", (size * gate * u).sum(0) * rows)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,d", CASES + [(3000, 136)])
def test_backward(T, d, kind, dtype):
    for seed, flags in enumerate([(1, 1, 1, 1, 1), (0, 1, 1, 0, 0), (1, 0, 0, 1, 1), (0, 0, 1, 1, 0),
                                  (1, 1, 1, 0, 0)]):
        post, pre, gate, scale, bias = flags
        a = _inputs(T, d, dtype, kind, post, pre, gate, scale, bias, seed=seed)
        _check_backward(a, kind, T, d, seed != 1, seed)
    a = _inputs(T, d, dtype, kind, 0, 1, 0, 0, 1, y=False)
    _check_backward(a, kind, T, d, True, 9)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_gradients_against_differences(kind):
    """Central differences of the forward pass itself, fp32: the loss is a sum of
    T d products, its differences over 2 h = 0.02 are good to a few 1e-3."""
    T, d, h = 6, 24, 1e-2
    a = _inputs(T, d, torch.float32, kind, 1, 1, 1, 1, 1)
    g = torch.Generator(device="cuda").manual_seed(3)
    dr, dh = (torch.randn((T, d), generator=g, device="cuda") for _ in range(2))

    def loss(b):
        o = swl.norm_residual(kind=kind, eps=EPS, **b)
        return float((o["r"].double() * dr + o["h"].double() * dh).sum())

    r = swl.norm_residual(kind=kind, eps=EPS, **a)["r"]
    got = swl.norm_residual_backward(dr, dh, r, kind=kind, eps=EPS,
                                     **{k: v for k, v in a.items() if k != "x"})
    for k, v in a.items():
        for at in range(0, v.numel(), max(1, v.numel() // 7)):
            if k == "y" and at // d % 7 == 0:
                continue                       # a zero row: its norm is not smooth on this scale
            b = [dict(a, **{k: v.clone()}) for _ in range(2)]
            b[0][k].view(-1)[at] += h
            b[1][k].view(-1)[at] -= h
            slope = (loss(b[0]) - loss(b[1])) / (2 * h)
            mine = float(got["d" + k].reshape(-1)[at])
            assert abs(slope - mine) <= 2e-2 * (1 + abs(mine)), (k, at)


def test_in_place_and_unaligned_and_repeatable():
    a = _inputs(50, 512, torch.bfloat16, "rms", 1, 1, 1, 1, 0)
    want = swl.norm_residual(eps=EPS, **a)
    x, y = a["x"].clone(), a["y"].clone()
    got = swl.norm_residual(eps=EPS, **dict(a, x=x, y=y), r=x, h=y)
    assert torch.equal(x, want["r"]) and torch.equal(y, want["h"]) and got["r"] is x
    # rows that start at an odd element: the same values by narrower loads
    flat = torch.empty(50 * 512 + 1, dtype=torch.bfloat16, device="cuda")
    x1 = flat[1:].view(50, 512)
    x1.copy_(a["x"])
    odd = swl.norm_residual(eps=EPS, **dict(a, x=x1))
    assert ((odd["r"].float() - want["r"].float()).abs() <= 2.0 ** -7 * want["r"].float().abs() + 1e-6).all()
    dr, dh = torch.randn_like(a["x"]), torch.randn_like(a["x"])
    args = {k: v for k, v in a.items() if k != "x"}
    one = swl.norm_residual_backward(dr, dh, want["r"], eps=EPS, **args)
    two = swl.norm_residual_backward(dr, dh, want["r"], eps=EPS, **args)
    for k in one:
        assert one[k] is None and two[k] is None or torch.equal(one[k], two[k]), k


def test_empty_batch_and_zero_and_non_finite_rows():
    a = _inputs(0, 64, torch.float32, "layer", 1, 1, 1, 1, 1)
    out = swl.norm_residual(kind="layer", eps=EPS, **a)
    assert out["r"].shape == (0, 64) and out["h"].shape == (0, 64)
    g = swl.norm_residual_backward(a["x"], a["x"].clone(), out["r"], kind="layer", eps=EPS,
                                   **{k: v for k, v in a.items() if k != "x"})
    for k in ("dw_pre", "db_pre", "dw_post", "db_post", "dscale"):
        assert (g[k] == 0).all()
    a = _inputs(40, 96, torch.float32, "rms", 1, 1, 1, 0, 0)
    a["x"][3] = 0
    a["y"][3] = 0
    a["x"][5, 7] = float("inf")
    a["x"][6, 7] = float("nan")
    out = swl.norm_residual(eps=EPS, **a)
    assert (out["h"][3] == 0).all() and (out["r"][3] == 0).all()
    assert out["h"][6].isnan().all()
    keep = [t for t in range(40) if t not in (5, 6)]
    assert torch.isfinite(out["h"][keep]).all() and torch.isfinite(out["r"][keep]).all()


def test_capture_and_side_stream():
    a = _inputs(200, 768, torch.bfloat16, "rms", 1, 1, 1, 1, 0)
    args = {k: v for k, v in a.items() if k != "x"}
    dr, dh = torch.randn_like(a["x"]), torch.randn_like(a["x"])
    want = swl.norm_residual(eps=EPS, **a)
    wantg = swl.norm_residual_backward(dr, dh, want["r"], eps=EPS, **args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = swl.norm_residual(eps=EPS, **a)
        g = swl.norm_residual_backward(dr, dh, out["r"], eps=EPS, **args)
    for _ in range(2):
        graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sg = swl.norm_residual_backward(dr, dh, want["r"], eps=EPS, stream=side, **args)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(out["r"], want["r"]) and torch.equal(out["h"], want["h"])
    for k in wantg:
        if wantg[k] is not None:
            assert torch.equal(g[k], wantg[k]) and torch.equal(sg[k], wantg[k]), k


def test_wrapper_refusals():
    a = _inputs(4, 32, torch.float32, "rms", 1, 1, 1, 1, 0)
    x = a["x"]
    for bad, err in ((dict(y=a["y"][:3]), ValueError), (dict(y=a["y"].bfloat16()), TypeError),
                     (dict(y=a["y"].t().contiguous().t()), ValueError),
                     (dict(w_pre=a["w_pre"].bfloat16()), TypeError),
                     (dict(gate=a["gate"].cpu()), ValueError), (dict(kind="batch"), ValueError),
                     (dict(eps=0.0), swl.SwitchLayerError), (dict(w_pre=None, h=x.clone()), ValueError),
                     (dict(b_pre=a["w_pre"]), swl.SwitchLayerError),
                     (dict(r=a["y"], h=a["y"]), swl.SwitchLayerError)):
        with pytest.raises(err):
            swl.norm_residual(**dict(a, **bad))
    with pytest.raises(swl.SwitchLayerError):
        swl.norm_residual(x)                                   # neither y nor w_pre
    with pytest.raises(swl.SwitchLayerError):
        swl.norm_residual(x, gate=a["gate"], w_pre=a["w_pre"])   # a gate without y
    wide = torch.zeros((1, 16385), device="cuda")
    with pytest.raises(swl.SwitchLayerError):
        swl.norm_residual(wide, w_pre=torch.ones(16385, device="cuda"))
    with pytest.raises(swl.SwitchLayerError):
        swl.norm_residual_backward(x, None, x, w_pre=a["w_pre"])   # dh is missing
