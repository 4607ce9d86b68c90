"""The rounding of the second moment's root in 8 bits, over the whole range of its codes.

Stochastic to three mantissa bits; e4m3 has fewer below 2^-6 of the scaled value, one spacing
of 2^-9 (a unit), and there the result is rounded to nearest.  Expectations are taken over
many equal elements, to five standard errors.
"""
from __future__ import annotations

import math

import pytest
import torch

import sparse_mixture_experts_argmax_b200 as swl
from sparse_mixture_experts_argmax_b200 import build as swl_build

pytestmark = pytest.mark.gpu

BLOCK = 256
UNIT = 2.0 ** -9


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    swl_build.build()
    swl.lib()


@pytest.mark.parametrize("units", [0.4, 1.0, 1.3, 1.4, 2.2, 3.4, 4.2, 5.6, 6.7, 7.9, 8.5, 12.25, 15.5, 17.0,
                                   30.5, 1000.0, 100000.0])
def test_the_root_is_rounded_as_stated(units):
    n = 1 << 17
    p = torch.zeros(n, device="cuda")
    grad = torch.full((n,), units * UNIT / 448, device="cuda")
    grad[::BLOCK] = 1.0                       # each block's largest: 448
    state = swl.adamw_state([p], 8)
    swl.adamw_step([p], [grad], state, lr=0.0, seed=4)
    r = state["v"][0].float().double().view(-1, BLOCK)[:, 1:] / UNIT
    step = 2.0 ** (math.floor(math.log2(units)) - 3)       # of three mantissa bits
    lo = step * math.floor(units / step)
    share = (units - lo) / step

    def code(v):                              # halves to even, and never zero
        return max(1.0, float(round(v))) if v < 8 else v

    a, b = code(lo), code(lo + step)
    assert ((r == a) | (r == b)).all()
    want, sd = a + share * (b - a), abs(b - a) * (share * (1 - share) / r.numel()) ** 0.5
    # the scaled root's own roundings, 8 of 2^-24, move the share and with it the mean
    assert abs(float(r.mean()) - want) <= 5 * sd + 8 * 2.0 ** -24 * units * max(1.0, (b - a) / step)
    if units >= 8:
        assert abs(want - units) <= 1e-9 * units            # unbiased


def test_a_root_at_the_small_end_may_stand_still():
    """What the interface says of it: from 4 units down without gradients, and one unit under
    gradients of up to 30, while one of 20 units fades and 8 grow."""
    b2, steps = 0.999, 300
    case = [(4, 0.0), (3, 0.0), (1, 29.0), (20, 0.0), (9, 60.0)]
    blocks = 256
    n = blocks * BLOCK
    p = torch.zeros(n, device="cuda")
    state = swl.adamw_state([p], 8)
    codes, grad = torch.full((blocks, BLOCK), UNIT, device="cuda"), torch.zeros((blocks, BLOCK), device="cuda")
    codes[:, 0], grad[:, 0] = 448.0, 1.0
    for i, (units, call) in enumerate(case):
        codes[:, 1 + 50 * i:51 + 50 * i] = units * UNIT
        grad[:, 1 + 50 * i:51 + 50 * i] = call * UNIT / 448
    state["v"][0].copy_(codes.view(-1).to(torch.float8_e4m3fn))
    state["v_scale"][0].fill_(1.0 / 448)
    for _ in range(steps):
        swl.adamw_step([p], [grad.view(-1)], state, lr=0.0, betas=(0.9, b2), seed=11)
    r = state["v"][0].float().view(blocks, BLOCK) / UNIT
    part = [r[:, 1 + 50 * i:51 + 50 * i] for i in range(len(case))]
    assert (part[0] == 4).all() and (part[1] == 3).all() and (part[2] == 1).all()
    kept = b2 ** steps
    # (12800 elements of a standard deviation under 3 units: 0.13 for the mean, and as much
    # again for the root's curvature, 3^2 / (8 r) of the mean square's spread at most a step)
    assert abs(float(part[3].mean()) - 20 * kept ** 0.5) < 0.5
    assert float(part[4].mean()) > 20
