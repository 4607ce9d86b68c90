"""The operators around the layer run together, as a training step uses them: the norm
before the block, the layer (or experts of the caller's own on the grouped products),
the norm after it with gate, residual scale and residual, the way back, and an AdamW
step over every tensor.

The gradients are compared with automatic differentiation of the formulas in 64 bits,
the routing taken from the layer.  Tolerance: whole tensors, normwise 1e-5 in fp32, the
one that the layer's own backward pass is held to (each tensor goes through fewer
than 10 products of at most 300 terms, sqrt(300) 2^-23 each if the roundings were all
to one side of independent signs, 2e-5 of the largest term and less of the norm).
"""
from __future__ import annotations

import pytest
import torch

import sparse_mixture_experts_argmax_b200 as swl
import synth
from sparse_mixture_experts_argmax_b200 import build as swl_build

pytestmark = pytest.mark.gpu

EPS = 1e-6
NORMWISE = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    swl_build.build()
    swl.lib()


def _hat(v):
    return v / (v.square().mean(1, keepdim=True) + EPS).sqrt()


def _same(got, want, what, size=None):
    """size: of the terms where a result is what is left of their cancellation."""
    err = float((got.double() - want).norm() / (want if size is None else size).norm().clamp(min=1e-30))
    assert err <= NORMWISE, (what, err)


def _block(seed, T, d, d_ff, N):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    p = {"w_in": 1 + n(d, std=0.1), "w_post": 1 + n(d, std=0.1), "w_next": 1 + n(d, std=0.1),
         "scale": 0.5 + n(d, std=0.1), "W_r": n(N, d, std=d ** -0.5), "b_r": n(N, std=0.1),
         "W1": n(N, d_ff, d, std=d ** -0.5), "b1": n(N, d_ff, std=0.1),
         "W2": n(N, d, d_ff, std=d_ff ** -0.5), "b2": n(N, d, std=0.1)}
    return p, n(T, d), n(T, d, std=0.1), n(T, d, std=0.1)


def _layer_step(p, x, dr, dh, cf):
    """Gradients of sum(dr r) + sum(dh h) for h0 = norm(x), y = layer(h0),
    r = x + scale norm(y), h = norm(r)."""
    T, d = x.shape
    N, d_ff, _ = p["W1"].shape
    h0 = swl.norm_residual(x, w_pre=p["w_in"], eps=EPS)["h"]
    inputs = {"x": h0, **{k: p[k] for k in ("W_r", "b_r", "W1", "b1", "W2", "b2")}}
    ws = swl.alloc_workspace(T, d, d_ff, N, x.dtype, cf)
    fwd = swl.forward(inputs, cf, workspace=ws, check=False)
    post = dict(y=fwd["out"], w_post=p["w_post"], scale=p["scale"], w_pre=p["w_next"], eps=EPS)
    out = swl.norm_residual(x, **post)
    g2 = swl.norm_residual_backward(dr, dh, out["r"], **post)
    gl = swl.backward(inputs, cf, fwd, ws, g2["dy"], check=False)
    g1 = swl.norm_residual_backward(g2["dx"], gl["dx"], x, w_pre=p["w_in"], eps=EPS)
    grads = {"w_in": g1["dw_pre"], "w_post": g2["dw_post"], "w_next": g2["dw_pre"],
             "scale": g2["dscale"], **{k: gl["d" + k] for k in ("W_r", "b_r", "W1", "b1", "W2", "b2")}}
    return fwd, out, grads, g1["dx"]


def test_layer_between_its_norms_and_an_optimiser_step():
    T, d, d_ff, N, cf = 257, 72, 96, 5, 1.0
    p, x, dr, dh = _block(1, T, d, d_ff, N)
    fwd, out, grads, dx = _layer_step(p, x, dr, dh, cf)
    D = {k: v.double().requires_grad_() for k, v in p.items()}
    X = x.double().requires_grad_()
    h0 = _hat(X) * D["w_in"]
    e = fwd["expert_idx"].long()
    prob = torch.softmax(h0 @ D["W_r"].T + D["b_r"], 1).gather(1, e[:, None])
    kept = fwd["pos_in_expert"] < swl.switch_layer_capacity(T, N, cf)
    assert 0 < int((~kept).sum()) < T                 # some tokens are dropped
    a = torch.relu(torch.einsum("tfd,td->tf", D["W1"][e], h0) + D["b1"][e])
    y = prob * (torch.einsum("tdf,tf->td", D["W2"][e], a) + D["b2"][e]) * kept[:, None]
    r = X + D["scale"] * (_hat(y) * D["w_post"])
    h = _hat(r) * D["w_next"]
    _same(out["r"], r.detach(), "r")
    _same(out["h"], h.detach(), "h")
    names = list(p)
    want = torch.autograd.grad((dr.double() * r).sum() + (dh.double() * h).sum(),
                               [X, y] + [D[k] for k in names])
    _same(dx, want[0], "dx")
    # The norm behind the layer takes the gate's size out again: of dout . out, which the
    # router's gradient dz_j = (dout . out) (delta_je - p_j) is made of, nothing but what
    # eps leaves remains.  Its error is that of the sum's terms.
    dot = (want[1].abs() * y.detach().abs()).sum(1, keepdim=True)
    p_all = torch.softmax(h0 @ D["W_r"].T + D["b_r"], 1).detach()
    dz = dot * (torch.nn.functional.one_hot(e, N) + p_all)
    sizes = {"W_r": dz.T @ h0.detach().abs(), "b_r": dz.sum(0)}
    for k, w in zip(names, want[2:]):
        _same(grads[k], w, k, sizes.get(k))
    # the step: every tensor moves by the rate against its gradient's sign (first step:
    # |m| / (sqrt(v) + eps) is 1 to 1e-3 for gradients of 1e-5 on, eps being 1e-8)
    before = {k: v.clone() for k, v in p.items()}
    state = swl.adamw_state([p[k] for k in names], 8)
    swl.adamw_step([p[k] for k in names], [grads[k] for k in names], state, lr=1e-3)
    for k in names:
        big = grads[k].abs() > 1e-5
        moved = (p[k] - before[k])[big]
        assert big.any() and ((moved + 1e-3 * grads[k][big].sign()).abs() <= 1e-3 * 1e-3 + 1e-6).all(), k


def _own_experts_step(p, x, dr, dh):
    """Experts of the caller's own, a gated unit without a capacity cut: the first
    product's 2 f features are a value and a gate."""
    T, d = x.shape
    N, two_f, _ = p["W1"].shape
    f = two_f // 2
    h0 = swl.norm_residual(x, w_pre=p["w_in"], eps=EPS)["h"]
    prob, e = torch.softmax(h0.float() @ p["W_r"].T + p["b_r"], 1).max(1)
    order = e.argsort(stable=True)
    offsets = torch.cat([e.new_zeros(1), torch.bincount(e, minlength=N).cumsum(0)]).to(torch.int32)
    rows = h0[order].contiguous()
    u = swl.grouped_matmul(rows, offsets, p["W1"], bias=p["b1"], check=False)
    act = (u[:, :f] * torch.sigmoid(u[:, f:])).contiguous()
    v = swl.grouped_matmul(act, offsets, p["W2"], bias=p["b2"], check=False)
    y = torch.empty_like(v)
    y[order] = v
    post = dict(y=y, gate=prob, w_post=p["w_post"], scale=p["scale"], w_pre=p["w_next"], eps=EPS)
    out = swl.norm_residual(x, **post)
    g = swl.norm_residual_backward(dr, dh, out["r"], **post)
    dv = g["dy"][order].contiguous()
    g2 = swl.grouped_matmul_backward(dv, act, offsets, p["W2"], check=False)
    s = torch.sigmoid(u[:, f:])
    du = torch.cat([g2["dx"] * s, g2["dx"] * u[:, :f] * s * (1 - s)], 1)
    g1 = swl.grouped_matmul_backward(du, rows, offsets, p["W1"], check=False)
    return e, out, {"w_post": g["dw_post"], "w_next": g["dw_pre"], "scale": g["dscale"],
                    "W1": g1["dW"], "b1": g1["db"], "W2": g2["dW"], "b2": g2["db"]}, g


def test_own_experts_on_the_grouped_products():
    T, d, f, N = 301, 80, 48, 6
    p, x, dr, dh = _block(2, T, d, 2 * f, N)
    p["W2"] = p["W2"][:, :, :f].contiguous()
    e, out, grads, g = _own_experts_step(p, x, dr, dh)
    D = {k: v.double().requires_grad_() for k, v in p.items()}
    X = x.double()
    h0 = _hat(X) * D["w_in"]
    prob = torch.softmax(h0 @ D["W_r"].T + D["b_r"], 1).gather(1, e[:, None])
    gate = prob.detach()[:, 0].requires_grad_()
    u = torch.einsum("tfd,td->tf", D["W1"][e], h0) + D["b1"][e]
    act = u[:, :f] * torch.sigmoid(u[:, f:])
    y = torch.einsum("tdf,tf->td", D["W2"][e], act) + D["b2"][e]
    r = X + gate[:, None] * D["scale"] * (_hat(y) * D["w_post"])
    h = _hat(r) * D["w_next"]
    _same(out["r"], r.detach(), "r")
    _same(out["h"], h.detach(), "h")
    names = list(grads)
    want = torch.autograd.grad((dr.double() * r).sum() + (dh.double() * h).sum(),
                               [gate] + [D[k] for k in names])
    _same(g["dgate"], want[0], "gate")
    for k, w in zip(names, want[1:]):
        _same(grads[k], w, k)


def test_captured_training_step_repeats_the_eager_one():
    T, d, d_ff, N, cf = 300, 64, 96, 4, 1.25
    p, x, dr, dh = _block(3, T, d, d_ff, N)
    p = {k: (v if k in ("w_in", "w_post", "w_next", "scale", "W_r", "b_r") else v.bfloat16())
         for k, v in p.items()}
    x, dr, dh = x.bfloat16(), dr.bfloat16(), dh.bfloat16()
    names = list(p)

    def step(p, state):
        _, _, grads, _ = _layer_step(p, x, dr, dh, cf)
        swl.adamw_step([p[k] for k in names], [grads[k] for k in names], state, lr=1e-3,
                       weight_decay=[0.1 if p[k].dim() > 1 else 0.0 for k in names], seed=5)

    eager = {k: v.clone() for k, v in p.items()}
    s0 = swl.adamw_state([eager[k] for k in names], 8, master=True)
    for _ in range(3):
        step(eager, s0)
    s1 = swl.adamw_state([p[k] for k in names], 8, master=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(p, s1)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert s1["step"].tolist() == [3, 0]
    for k in names:
        assert torch.isfinite(p[k].float()).all()
        # (the layer's aux-loss sums run in an order of their own; everything else repeats)
        assert ((p[k].float() - eager[k].float()).abs() <= 2e-3 + 2.0 ** -7 * p[k].float().abs()).all(), k
