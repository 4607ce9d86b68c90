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
