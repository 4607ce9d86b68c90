"""switch_layer_adamw_step against the step's formulas in 64 bits.

u = 2^-24 is half a step of fp32.  Each of the kernel's operations is rounded
once, so (with the constants' own roundings) m is off by at most 6 u of the sizes
of its two terms, v by at most 8 u of itself, the denominator by 10 u with its root, the quotient by
16 u with the division, and the weight by the update's share of these plus 3 u of
its own size.
"""
from __future__ import annotations

import pytest
import torch

import sparse_mixture_experts_argmax_b200 as swl
from sparse_mixture_experts_argmax_b200 import build as swl_build

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BLOCK = 256
LR, B1, B2, EPS = 2e-3, 0.9, 0.999, 1e-8
TYPES = {"f32": (torch.float32, False), "bf16": (torch.bfloat16, False),
         "bf16_master": (torch.bfloat16, True)}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    swl_build.build()
    swl.lib()


def _blocks(t):
    """[blocks, 256], the last block filled with zeros."""
    n = t.numel()
    return torch.nn.functional.pad(t.reshape(-1), (0, -n % BLOCK)).view(-1, BLOCK)


def _decoded(state, i):
    m, v = state["m"][i], state["v"][i]
    if state["m_scale"][i] is None:
        return m.double(), v.double()
    n = m.numel()
    dm = _blocks(m.float()).double() * state["m_scale"][i].double()[:, None]
    dr = _blocks(v.float()).double() * state["v_scale"][i].double()[:, None]
    return dm.reshape(-1)[:n], dr.reshape(-1)[:n].square()


def _clone(state):
    return {k: (v.clone() if k == "step" else [None if t is None else t.clone() for t in v])
            for k, v in state.items()}


def _check_step(params0, grads, s0, params, s1, wd, gs=1.0, lrs=1.0):
    """One step from (params0, s0) to (params, s1)."""
    t = int(s0["step"][0]) + 1
    assert s1["step"].tolist() == [t, 0]
    lr = LR * lrs
    for i, (p0, g, p1) in enumerate(zip(params0, grads, params)):
        if p0.numel() == 0:
            continue
        g = g.double().reshape(-1) * gs
        w0 = (p0 if s0["master"][i] is None else s0["master"][i]).double().reshape(-1)
        m0, v0 = _decoded(s0, i)
        m = B1 * m0 + (1 - B1) * g
        v = B2 * v0 + (1 - B2) * g * g
        em = 6 * U * (B1 * m0.abs() + (1 - B1) * g.abs())
        root = (v / (1 - B2 ** t)).sqrt() + EPS
        rate = lr / (1 - B1 ** t)
        w = w0 * (1 - lr * wd[i]) - rate * m / root
        ew = rate * (em / root + 16 * U * m.abs() / root) + 3 * U * (w0.abs() + w.abs()) + 1e-38
        if s0["master"][i] is not None:
            assert ((s1["master"][i].double() - w).abs() <= ew).all(), i
        half = 2.0 ** -8 * w.abs() if p1.dtype == torch.bfloat16 else 0.0
        assert ((p1.double().reshape(-1) - w).abs() <= ew + half + 1e-40).all(), i
        m1, v1 = _decoded(s1, i)
        if s0["m_scale"][i] is None:
            assert ((m1 - m).abs() <= em + 1e-44).all(), i
            assert ((v1 - v).abs() <= 8 * U * v + 1e-44).all(), i
            continue
        top_m, top_r = _blocks(m).abs().amax(1), _blocks(v).sqrt().amax(1)
        assert ((s1["m_scale"][i].double() - top_m / 448).abs() <= 8 * U * top_m / 448).all()
        assert ((s1["v_scale"][i].double() - top_r / 448).abs() <= 8 * U * top_r / 448).all()
        # m: half a spacing of e4m3 (2^-4 of the value, at least half of 2^-9 of the scale);
        # the root: less than one spacing, and never zero
        wide_m = top_m.repeat_interleave(BLOCK)[:m.numel()] / 448
        wide_r = top_r.repeat_interleave(BLOCK)[:m.numel()] / 448
        assert ((m1 - m).abs() <= (2.0 ** -4 * m.abs()).maximum(2.0 ** -10 * wide_m) * (1 + 1e-5)).all()
        r, r1 = v.sqrt(), v1.sqrt()
        assert ((r1 - r).abs() <= (2.0 ** -3 * r).maximum(2.0 ** -9 * wide_r) * (1 + 1e-5)).all()
        assert (r1[r > 0] > 0).all()


def _make(sizes, dtype, g, std=0.05):
    return [(torch.randn(n, generator=g, device="cuda") * std).to(dtype) for n in sizes]


SIZES = [1, 3, 255, 256, 257, 0, 4096, 4099, 70001]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kind", list(TYPES))
def test_steps_match_formulas(kind, bits):
    dtype, master = TYPES[kind]
    g = torch.Generator(device="cuda").manual_seed(bits)
    params = _make(SIZES, dtype, g)
    wd = [0.1 * (i % 2) for i in range(len(SIZES))]
    state = swl.adamw_state(params, bits, master)
    for step in range(3):
        grads = _make(SIZES, dtype, g, 10.0 ** -step)
        gs = torch.full((1,), 0.25, device="cuda") if step == 1 else None
        ls = torch.full((1,), 0.5, device="cuda") if step == 2 else None
        p0, s0 = [p.clone() for p in params], _clone(state)
        swl.adamw_step(params, grads, state, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=wd,
                       grad_scale=gs, lr_scale=ls, seed=3)
        _check_step(p0, grads, s0, params, state, wd, 1.0 if gs is None else 0.25,
                    1.0 if ls is None else 0.5)


@pytest.mark.parametrize("bits", [32, 8])
def test_mixed_types_and_more_tensors_than_one_launch(bits):
    g = torch.Generator(device="cuda").manual_seed(5)
    sizes = [1 + 37 * i % 700 for i in range(333)]
    params = [_make([n], torch.bfloat16 if i % 3 else torch.float32, g)[0]
              for i, n in enumerate(sizes)]
    grads = [torch.randn(p.shape, generator=g, device="cuda").to(p.dtype) for p in params]
    state = swl.adamw_state(params, bits, master=True)
    p0, s0 = [p.clone() for p in params], _clone(state)
    before = swl.switch_layer_launch_count()
    swl.adamw_step(params, grads, state, lr=LR, betas=(B1, B2), eps=EPS)
    assert swl.switch_layer_launch_count() - before == 3    # 222 of one kind, 111 of the other
    _check_step(p0, grads, s0, params, state, [0.0] * len(sizes))


def test_capture_counts_its_replays_and_repeats_bit_for_bit():
    g = torch.Generator(device="cuda").manual_seed(6)
    params = _make([5000, 300], torch.bfloat16, g)
    grads = _make([5000, 300], torch.bfloat16, g, 1.0)
    state = swl.adamw_state(params, 8, master=True)
    pe, se = [p.clone() for p in params], _clone(state)
    for _ in range(3):
        swl.adamw_step(pe, grads, se, lr=LR, seed=9)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        swl.adamw_step(params, grads, state, lr=LR, seed=9)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert state["step"].tolist() == [3, 0]
    for k in range(2):
        assert torch.equal(params[k], pe[k]) and torch.equal(state["master"][k], se["master"][k])
        for s in ("m", "v"):
            assert torch.equal(state[s][k].view(torch.uint8), se[s][k].view(torch.uint8))


def test_rounding_of_the_root_has_no_drift():
    """The root's stochastic rounding is unbiased: over 2^17 equal elements its
    mean is the unrounded root to within five standard errors (a spacing of 32
    codes, a binomial share p: sd = 32 sqrt(p (1 - p) / n))."""
    n = 1 << 17
    p = torch.zeros(n, device="cuda")
    grad = torch.full((n,), 0.83, device="cuda")
    grad[::BLOCK] = 1.0                       # each block's largest
    state = swl.adamw_state([p], 8)
    swl.adamw_step([p], [grad], state, lr=0.0, seed=1)
    r = state["v"][0].float().double().view(-1, BLOCK)[:, 1:]
    q = 0.83 * 448
    lo, hi = 352.0, 384.0
    assert ((r == lo) | (r == hi)).all()
    share = (q - lo) / (hi - lo)
    sd = (hi - lo) * (share * (1 - share) / r.numel()) ** 0.5
    assert abs(float(r.mean()) - q) < 5 * sd
    again = swl.adamw_state([p], 8)
    swl.adamw_step([p], [grad], again, lr=0.0, seed=2)
    assert not torch.equal(again["v"][0].view(torch.uint8), state["v"][0].view(torch.uint8))


def test_zero_and_tiny_blocks_and_non_finite_gradients():
    p = torch.zeros(4 * BLOCK, device="cuda")
    grad = torch.zeros(4 * BLOCK, device="cuda")
    grad[BLOCK:2 * BLOCK] = 1e-33             # m under 2^-100: held as zeros
    grad[2 * BLOCK + 5] = float("nan")
    grad[3 * BLOCK + 5] = 1.0
    state = swl.adamw_state([p], 8)
    swl.adamw_step([p], [grad], state, lr=LR)
    m, v = _decoded(state, 0)
    m, v, w = m.view(4, -1), v.view(4, -1), p.view(4, -1)
    assert (m[:2] == 0).all() and (v[:2] == 0).all() and (w[0] == 0).all()
    assert m[2].isnan().all() and v[2].isnan().all()
    assert w[2].isnan().sum() == 1 and w[2, 5].isnan()
    assert m[3].count_nonzero() == 1 and torch.isfinite(w[3]).all()
    for bad in (float("inf"), float("nan")):
        p = torch.zeros(300, device="cuda")
        grad = torch.zeros(300, device="cuda")
        grad[7] = bad
        state = swl.adamw_state([p], 32)
        swl.adamw_step([p], [grad], state, lr=LR)
        assert not torch.isfinite(state["m"][0][7]) and not torch.isfinite(p[7])
        assert torch.isfinite(p[8:]).all() and torch.isfinite(p[:7]).all()


def test_offsets_past_32_bits():
    n = (1 << 31) + 259
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    grad = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    grad[-259:] = torch.linspace(0.1, 1.0, 259, device="cuda").bfloat16()
    state = swl.adamw_state([p], 8)
    swl.adamw_step([p], [grad], state, lr=LR)
    tail = [p[-259:].clone()], [grad[-259:].clone()]
    p1 = [torch.zeros(259, dtype=torch.bfloat16, device="cuda")]
    s1 = swl.adamw_state(p1, 8)
    swl.adamw_step(p1, tail[1], s1, lr=LR)
    assert torch.equal(tail[0][0], p1[0])
    assert torch.equal(state["m_scale"][0][-2:], s1["m_scale"][0])
    # the first moment's bytes (the root's rounding bits differ by position)
    assert torch.equal(state["m"][0][-259:].view(torch.uint8), s1["m"][0].view(torch.uint8))
    assert (p[:1 << 20] == p[0]).all() and p[0] != 0


def test_side_stream_and_wrapper_refusals():
    g = torch.Generator(device="cuda").manual_seed(8)
    params = _make([1000], torch.float32, g)
    grads = _make([1000], torch.float32, g)
    state = swl.adamw_state(params)
    p0, s0 = [p.clone() for p in params], _clone(state)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    swl.adamw_step(params, grads, state, lr=LR, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    _check_step(p0, grads, s0, params, state, [0.0])
    with pytest.raises(swl.SwitchLayerError):          # the same tensor twice
        swl.adamw_step(params * 2, grads * 2, {k: (v if k == "step" else v * 2)
                                               for k, v in state.items()})
    with pytest.raises(swl.SwitchLayerError):          # a gradient that is the parameter
        swl.adamw_step(params, params, state)
    with pytest.raises(swl.SwitchLayerError):          # not 16-byte aligned
        swl.adamw_step([params[0][1:]], [grads[0][1:]], swl.adamw_state([params[0][1:]]))
    with pytest.raises(ValueError):
        swl.adamw_step(params, [grads[0][:-1]], state)
    with pytest.raises(ValueError):
        swl.adamw_step([params[0].view(500, 2).t()], grads, state)
    with pytest.raises(TypeError):
        swl.adamw_step([params[0].half()], [grads[0].half()], state)
    assert state["step"].tolist() == [1, 0]
