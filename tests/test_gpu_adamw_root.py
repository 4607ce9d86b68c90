"""The rounding of the second moment's root in 8 bits at the small end of its codes.

Below 2^-6 of the scaled value e4m3 has one spacing, 2^-9 (a unit): the stochastic
rounding has to be to that grid, or a root of a few units never moves.  Expectations are
taken over many equal elements, to five standard errors.
"""
from __future__ import annotations

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


@pytest.mark.parametrize("units", [0.4, 1.0, 1.3, 2.2, 3.4, 5.6, 6.7, 7.5, 8.5, 12.25, 15.5, 17.0, 30.5])
def test_the_root_is_unbiased_on_the_grid_of_its_codes(units):
    n = 1 << 17
    p = torch.zeros(n, device="cuda")
    grad = torch.full((n,), units * UNIT / 448, device="cuda")
    grad[::BLOCK] = 1.0                       # each block's largest: 448
    state = swl.adamw_state([p], 8)
    swl.adamw_step([p], [grad], state, lr=0.0, seed=4)
    r = state["v"][0].float().double().view(-1, BLOCK)[:, 1:] / UNIT
    if units <= 1:                            # a root that is not zero keeps the smallest code
        assert (r == 1).all()
        return
    step = 1 if units < 16 else 2             # 2^-6 is 8 units, 2^-5 is 16
    lo = step * (units // step)
    assert ((r == lo) | (r == lo + step)).all()
    share = (units - lo) / step
    # the scaled root's own roundings (8 of 2^-24, of values up to 32) shift the mean by 2e-5
    sd = step * (share * (1 - share) / r.numel()) ** 0.5
    assert abs(float(r.mean()) - units) <= 5 * sd + 2e-5


def _mean_units(units, grad_units, b2, steps):
    """Mean and standard deviation of a root after some steps: the chain over whole units
    whose step rounds sqrt(b2 r^2 + (1 - b2) g^2) to one of its two neighbours without bias."""
    p = torch.zeros(17, dtype=torch.float64)
    p[units] = 1.0
    r = torch.arange(17, dtype=torch.float64)
    to = (b2 * r.square() + (1 - b2) * grad_units ** 2).sqrt().clamp(1, 15.5)
    lo = to.floor().long()
    share = to - lo
    for _ in range(steps):
        p = torch.zeros_like(p).scatter_add_(0, lo, p * (1 - share)).scatter_add_(0, lo + 1, p * share)
    mean = float((p * r).sum())
    return mean, float((p * (r - mean).square()).sum()) ** 0.5


def test_a_small_root_follows_its_gradients():
    """A root of 6 units whose gradients have gone away, and one of 2 units whose gradients
    call for 6, over 400 steps beside a large element that stays."""
    blocks, steps, b2 = 512, 400, 0.999
    n = blocks * BLOCK
    p = torch.zeros(n, device="cuda")
    state = swl.adamw_state([p], 8)
    codes = torch.full((blocks, BLOCK), 6 * UNIT, device="cuda")
    codes[:, 129:] = 2 * UNIT
    codes[:, 0] = 448.0
    state["v"][0].copy_(codes.view(-1).to(torch.float8_e4m3fn))
    state["v_scale"][0].fill_(1.0 / 448)
    grad = torch.zeros((blocks, BLOCK), device="cuda")
    grad[:, 129:] = 6 * UNIT / 448
    grad[:, 0] = 1.0
    for _ in range(steps):
        swl.adamw_step([p], [grad.view(-1)], state, lr=0.0, betas=(0.9, b2), seed=11)
    r = (state["v"][0].float().view(blocks, BLOCK).double() *
         state["v_scale"][0].double()[:, None]) * 448 / UNIT
    # the largest root: sqrt(b2 + (1 - b2)) = 1, 10 roundings of 2^-24 a step
    assert ((r[:, 0] * UNIT / 448 - 1).abs() <= steps * 10 * 2.0 ** -24).all()
    for got, first, call in ((r[:, 1:129], 6, 0.0), (r[:, 129:], 2, 6.0)):
        mean, sd = _mean_units(first, call, b2, steps)
        # (the largest root's drift, as above, and as much again for the small one's roundings)
        assert abs(float(got.mean()) - mean) <= 5 * sd / got.numel() ** 0.5 + \
            2 * steps * 10 * 2.0 ** -24 * mean, (first, float(got.mean()), mean, sd)
