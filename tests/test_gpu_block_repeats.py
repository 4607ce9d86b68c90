"""A training step of the block (norm, layer, norm, the way back, AdamW) captured into a
graph gives what the eager one gives, bit for bit: every sum on the way to a gradient runs in
a fixed order (the auxiliary loss's own sums, which nothing here takes a gradient of, aside)."""
from __future__ import annotations

import pytest
import torch

import sparse_mixture_experts_argmax_b200 as swl
from sparse_mixture_experts_argmax_b200 import build as swl_build
from test_gpu_block import _block, _layer_step, _own_experts_step

pytestmark = pytest.mark.gpu

FP32 = ("w_in", "w_post", "w_next", "scale", "W_r", "b_r")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    swl_build.build()
    swl.lib()


def _bits(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t


def _same(a, b, sa, sb, names):
    for k in names:
        assert torch.equal(a[k], b[k]), k
    for key in ("m", "v", "m_scale", "v_scale", "master"):
        for k, x, y in zip(names, sa[key], sb[key]):
            assert (x is None) == (y is None) and (x is None or torch.equal(_bits(x), _bits(y))), (key, k)
    assert torch.equal(sa["step"], sb["step"])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", ["layer", "own experts"])
def test_captured_steps_repeat_eager_ones_bit_for_bit(kind, dtype):
    T, d, d_ff, N = 300, 64, 96, 4
    p, x, dr, dh = _block(3, T, d, d_ff, N)
    if kind == "own experts":
        p["W2"] = p["W2"][:, :, :d_ff // 2].contiguous()
    p = {k: v if k in FP32 else v.to(dtype) for k, v in p.items()}
    x, dr, dh = x.to(dtype), dr.to(dtype), dh.to(dtype)

    def gradients(p):
        if kind == "layer":
            return _layer_step(p, x, dr, dh, 1.25)[2]
        return _own_experts_step(p, x, dr, dh)[2]

    names = list(gradients(p))

    def step(p, state):
        grads = gradients(p)
        swl.adamw_step([p[k] for k in names], [grads[k] for k in names], state, lr=1e-3,
                       weight_decay=[0.1 if p[k].dim() > 1 else 0.0 for k in names], seed=5)

    def fresh():
        q = {k: v.clone() for k, v in p.items()}
        return q, swl.adamw_state([q[k] for k in names], 8, master=True)

    eager, s0 = fresh()
    for _ in range(3):
        step(eager, s0)
    again, s1 = fresh()
    for _ in range(3):
        step(again, s1)
    _same(eager, again, s0, s1, names)
    captured, s2 = fresh()
    if kind == "layer":
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(captured, s2)
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        _same(eager, captured, s0, s2, names)
    assert any(not torch.equal(eager[k], p[k]) for k in names)
