"""Host-side checks of the operators around the layer: refusals are made before
anything is enqueued.  No kernel is launched here (the pointers are invented)."""
import ctypes

import pytest

import sparse_mixture_experts_argmax_b200 as swl
from sparse_mixture_experts_argmax_b200 import build as swl_build

OK, INVALID, UNSUPPORTED, WORKSPACE, CUDA = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    swl_build.build()
    return swl.lib()


# ---------------------------------------------------------------- AdamW
def _adamw(L, change=None, tensors=1, cfg=None, step=0x100000, grad_scale=None, lr_scale=None):
    table = (swl.AdamwTensor * max(1, tensors))()
    for i in range(tensors):
        at = 0x1000000 * (i + 1)
        e = dict(n=1000, dtype=swl.SWL_BF16, state_bits=8, weight_decay=0.1, param=at,
                 grad=at + 0x10000, m=at + 0x20000, v=at + 0x30000, m_scale=at + 0x40000,
                 v_scale=at + 0x50000, master=at + 0x60000)
        if i == tensors - 1:
            e.update(change or {})
        table[i] = swl.AdamwTensor(**e)
    c = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, seed=0)
    c.update(cfg or {})
    before = L.switch_layer_launch_count()
    st = L.switch_layer_adamw_step(table, tensors, ctypes.byref(swl.Adamw(**c)), step, grad_scale,
                                   lr_scale, None)
    assert L.switch_layer_launch_count() == before
    return st


@pytest.mark.parametrize("change", [
    dict(n=-1), dict(dtype=7), dict(state_bits=16), dict(weight_decay=-1.0),
    dict(weight_decay=float("nan")), dict(param=None), dict(grad=None), dict(m=None),
    dict(v=None), dict(m_scale=None), dict(v_scale=None), dict(state_bits=32),
    dict(dtype=swl.SWL_F32),                             # a master of an fp32 parameter
    dict(m=0x1000400), dict(v=0x1000000),          # written twice
    dict(grad=0x1000400),                                 # a gradient inside the parameter
    dict(v_scale=0x1040000), dict(m=0x100000),            # the scales, the step
], ids=str)
def test_adamw_refuses_invalid_tensors(L, change):
    assert _adamw(L, change) == INVALID


def test_adamw_refuses_a_tensor_listed_twice(L):
    assert _adamw(L, dict(param=0x1000000), tensors=2) == INVALID
    assert _adamw(L, dict(grad=0x1060000), tensors=2) == INVALID   # the first one's master
    assert _adamw(L, grad_scale=0x1000000) == INVALID
    assert _adamw(L, lr_scale=0x100004) == INVALID


@pytest.mark.parametrize("change", [dict(param=0x1000002), dict(grad=0x1010008),
                                    dict(m=0x1020004), dict(v=0x1030001), dict(master=0x1060008),
                                    dict(m_scale=0x1040002), dict(v_scale=0x1050001),
                                    dict(n=1 << 41)], ids=str)
def test_adamw_refuses_unsupported_tensors(L, change):
    assert _adamw(L, change) == UNSUPPORTED


def test_adamw_refuses_bad_calls(L):
    for cfg in (dict(lr=-1.0), dict(lr=float("inf")), dict(beta1=1.0), dict(beta2=-0.1),
                dict(beta2=float("nan")), dict(eps=0.0), dict(eps=-1.0), dict(eps=1e-60)):
        assert _adamw(L, cfg=cfg) == INVALID, cfg
    assert _adamw(L, step=None) == INVALID
    assert _adamw(L, step=0x100004) == UNSUPPORTED
    assert _adamw(L, grad_scale=0x200002) == UNSUPPORTED
    assert L.switch_layer_adamw_step(None, 1, ctypes.byref(swl.Adamw(1e-3, .9, .9, 1e-8, 0)),
                                     0x100000, None, None, None) == INVALID
    assert L.switch_layer_adamw_step(None, 0, None, 0x100000, None, None, None) == INVALID


# ---------------------------------------------------------------- norms around a block
def _norm(L, T=4, d=64, dtype=swl.SWL_BF16, kind=0, eps=1e-6, change=None, norm=None):
    a = dict(x=0x10000, y=0x20000, gate=0x30000, r=0x40000, h=0x50000)
    n = dict(w_pre=0x61000, w_post=0x62000, scale=0x63000)
    a.update(change or {})
    n.update(norm or {})
    s = swl.Norm(kind, eps, n.get("w_pre"), n.get("b_pre"), n.get("w_post"), n.get("b_post"),
                 n.get("scale"))
    before = L.switch_layer_launch_count()
    st = L.switch_layer_norm_residual(T, d, dtype, a["x"], a["y"], a["gate"], ctypes.byref(s),
                                      a["r"], a["h"], None)
    assert L.switch_layer_launch_count() == before
    return st


def test_norm_residual_refusals(L):
    for kw in (dict(T=-1), dict(d=0), dict(dtype=5), dict(kind=2), dict(eps=0.0),
               dict(eps=float("nan")), dict(norm=dict(b_pre=0x64000)), dict(change=dict(x=None)),
               dict(change=dict(r=None)), dict(change=dict(y=None)), dict(change=dict(h=None)),
               dict(norm=dict(w_pre=None)), dict(change=dict(r=0x50000)),      # r is h
               dict(change=dict(r=0x10100)), dict(change=dict(h=0x20002)),     # across x, y
               dict(change=dict(h=0x61000)), dict(change=dict(r=0x30000)),     # on w_pre, gate
               dict(kind=1, norm=dict(w_post=None, b_post=0x64000))):
        assert _norm(L, **kw) == INVALID, kw
    for kw in (dict(d=16385), dict(change=dict(x=0x10001)), dict(change=dict(gate=0x30002)),
               dict(norm=dict(scale=0x63002)), dict(dtype=swl.SWL_F32, change=dict(h=0x50002))):
        assert _norm(L, **kw) == UNSUPPORTED, kw
    assert L.switch_layer_norm_residual(4, 64, 1, 0x10000, None, None, None, None, 0x50000,
                                        None) == INVALID
    assert _norm(L, T=0) == OK                       # an empty batch: nothing to do


def _norm_bwd(L, T=4, d=64, change=None, norm=None, out=None, ws=0x100000, ws_bytes=1 << 20,
              kind=0):
    a = dict(dr=0x10000, dh=0x11000, r=0x12000, y=0x13000, gate=0x14000)
    n = dict(w_pre=0x21000, w_post=0x22000, scale=0x23000)
    o = dict(dx=0x30000, dy=0x31000, dgate=0x32000, dw_pre=0x33000, dw_post=0x34000,
             dscale=0x35000)
    a.update(change or {})
    n.update(norm or {})
    o.update(out or {})
    s = swl.Norm(kind, 1e-6, n.get("w_pre"), n.get("b_pre"), n.get("w_post"), n.get("b_post"),
                 n.get("scale"))
    g = swl.NormGrads(**o)
    before = L.switch_layer_launch_count()
    st = L.switch_layer_norm_residual_backward(T, d, 1, a["dr"], a["dh"], a["r"], a["y"],
                                               a["gate"], ctypes.byref(s), ctypes.byref(g), ws,
                                               ws_bytes, None)
    assert L.switch_layer_launch_count() == before
    return st


def test_norm_residual_backward_refusals(L):
    for kw in (dict(change=dict(dh=None)), dict(change=dict(r=None)), dict(out=dict(dx=None)),
               dict(out=dict(dy=None)), dict(change=dict(y=None)), dict(norm=dict(w_pre=None)),
               dict(change=dict(gate=None)), dict(out=dict(db_pre=0x36000)),
               dict(norm=dict(scale=None)), dict(ws=None), dict(out=dict(dy=0x30000)),
               dict(out=dict(dx=0x11000)), dict(out=dict(dx=0x10002)), dict(out=dict(dscale=0x33004)),
               dict(out=dict(dw_pre=0x21000)), dict(ws=0x12000), dict(out=dict(dgate=0x14000)),
               dict(norm=dict(w_pre=None, w_post=None, scale=None),
                    change=dict(dr=None, dh=None), out=dict(dw_pre=None, dw_post=None, dscale=None))):
        assert _norm_bwd(L, **kw) == INVALID, kw
    for kw in (dict(d=20000), dict(change=dict(dr=0x10001)), dict(out=dict(dw_pre=0x33002)),
               dict(ws=0x100010)):
        assert _norm_bwd(L, **kw) == UNSUPPORTED, kw
    assert _norm_bwd(L, ws_bytes=64) == WORKSPACE
    n = ctypes.c_size_t()
    size = L.switch_layer_norm_residual_backward_workspace_size
    assert size(10, 64, 1, ctypes.byref(n)) == OK and n.value == 10 * 5 * 64 * 4
    assert size(1 << 30, 64, 1, ctypes.byref(n)) == OK and n.value < 1 << 20
    assert size(10, 64, 1, None) == INVALID and size(10, 1 << 20, 0, ctypes.byref(n)) == UNSUPPORTED


# ---------------------------------------------------------------- grouped products
def _grouped(L, R=100, K=64, O=128, N=4, dtype=swl.SWL_BF16, change=None, ws_bytes=1 << 20):
    a = dict(x=0x100000, off=0x200000, W=0x300000, bias=0x400000, y=0x500000, ws=0x600000)
    a.update(change or {})
    before = L.switch_layer_launch_count()
    st = L.switch_layer_grouped_matmul(R, K, O, N, dtype, a["x"], a["off"], a["W"], a["bias"],
                                       a["y"], a["ws"], ws_bytes, None)
    assert L.switch_layer_launch_count() == before
    return st


def _grouped_bwd(L, R=100, K=64, O=128, N=4, dtype=swl.SWL_BF16, change=None, ws_bytes=1 << 20):
    a = dict(dy=0x080000, x=0x100000, off=0x200000, W=0x300000, dx=0x400000, dW=0x500000,
             db=0x600000, ws=0x700000)
    a.update(change or {})
    before = L.switch_layer_launch_count()
    st = L.switch_layer_grouped_matmul_backward(R, K, O, N, dtype, a["dy"], a["x"], a["off"],
                                                a["W"], a["dx"], a["dW"], a["db"], a["ws"],
                                                ws_bytes, None)
    assert L.switch_layer_launch_count() == before
    return st


@pytest.mark.parametrize("call", [_grouped, _grouped_bwd], ids=["forward", "backward"])
def test_grouped_refusals(L, call):
    for kw in (dict(R=-1), dict(K=0), dict(O=0), dict(N=0), dict(dtype=3),
               dict(change=dict(x=None)), dict(change=dict(off=None)), dict(change=dict(W=None)),
               dict(change=dict(ws=None))):
        assert call(L, **kw) == INVALID, kw
    for kw in (dict(K=12), dict(O=20), dict(N=1 << 21), dict(R=1 << 31), dict(N=1 << 18, K=1 << 14),
               dict(change=dict(x=0x100008)), dict(change=dict(W=0x300002)),
               dict(change=dict(off=0x200002)), dict(change=dict(ws=0x600080)),
               dict(dtype=swl.SWL_F32, change=dict(x=0x100002)), dict(R=1 << 29, K=1 << 13, O=8)):
        assert call(L, **kw) == UNSUPPORTED, kw
    assert call(L, ws_bytes=256) == WORKSPACE


def test_grouped_refuses_overlaps(L):
    for change in (dict(y=0x100000), dict(y=0x300100), dict(y=0x400010 - 0x10), dict(ws=0x500100),
                   dict(y=0x200000), dict(y=None)):
        assert _grouped(L, change=change) == INVALID, change
    for change in (dict(dx=0x080000), dict(dx=0x100000), dict(dW=0x300000), dict(dx=0x500000),
                   dict(db=0x500002), dict(ws=0x400000), dict(dy=None),
                   dict(dx=None, dW=None, db=None)):
        assert _grouped_bwd(L, change=change) == INVALID, change


def test_grouped_workspace_size(L):
    n = swl.switch_layer_grouped_workspace_size(1000, 64, 128, 2048, swl.SWL_BF16)
    assert n >= 2049 * 4 + 256
    with pytest.raises(swl.SwitchLayerError) as e:
        swl.switch_layer_grouped_workspace_size(10, 12, 128, 4, swl.SWL_BF16)
    assert e.value.status == UNSUPPORTED
    assert L.switch_layer_grouped_workspace_size(10, 8, 8, 4, 1, None) == INVALID
