"""Finite values whose squares pass fp32's range stay in their rows and blocks, as the
interface says."""
from __future__ import annotations

import pytest
import torch

import sparse_mixture_experts_argmax_b200 as swl
from sparse_mixture_experts_argmax_b200 import build as swl_build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    swl_build.build()
    swl.lib()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norms_of_rows_past_the_range(kind, dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    T, d = 40, 72
    x = torch.randn((T, d), generator=g, device="cuda").to(dtype)
    y = torch.randn((T, d), generator=g, device="cuda").to(dtype)
    w = 1 + torch.randn(d, generator=g, device="cuda")
    dr, dh = (torch.randn((T, d), generator=g, device="cuda").to(dtype) for _ in range(2))
    args = dict(w_pre=w, w_post=w, kind=kind)
    want = swl.norm_residual(x, y=y, **args)
    wantg = swl.norm_residual_backward(dr, dh, want["r"], y=y, **args)
    lowest = -torch.finfo(dtype).max
    x[7], x[20, 3], y[30] = lowest, 1e25, lowest
    got = swl.norm_residual(x, y=y, **args)
    r = got["r"].clone()
    r[[7, 20, 30]] = want["r"][[7, 20, 30]]
    rest = [t for t in range(T) if t not in (7, 20, 30)]
    assert torch.equal(got["r"][rest], want["r"][rest]) and torch.equal(got["h"][rest], want["h"][rest])
    assert torch.equal(r, want["r"])
    if kind == "rms":
        assert (got["h"][[7, 20]] == 0).all()
    gg = swl.norm_residual_backward(dr, dh, got["r"], y=y, **args)
    for k in ("dx", "dy"):
        assert torch.equal(gg[k][rest], wantg[k][rest]), k


def test_adamw_of_gradients_past_the_range():
    g = torch.Generator(device="cuda").manual_seed(2)
    n = 3 * 256
    grad = torch.randn(n, generator=g, device="cuda")
    grad[300] = 2.0 ** 64
    for bits in (32, 8):
        p, q = torch.ones(n, device="cuda"), torch.ones(n, device="cuda")
        a, b = swl.adamw_state([p], bits), swl.adamw_state([q], bits)
        plain = grad.clone()
        plain[300] = 0
        for _ in range(3):
            swl.adamw_step([p], [grad], a, lr=1e-2, weight_decay=0.5)
            swl.adamw_step([q], [plain], b, lr=1e-2, weight_decay=0.5)
        rest = torch.ones(n, dtype=torch.bool, device="cuda")
        if bits == 32:
            rest[300] = False
            # three decays of 1 - 0.005, a rounding of the factor and one of each product
            assert abs(float(p[300]) - 0.995 ** 3) <= 6 * 2.0 ** -24
        else:
            rest[256:512] = False
            assert not torch.isfinite(a["v_scale"][0][1]) and torch.isfinite(a["v_scale"][0][[0, 2]]).all()
        assert torch.equal(p[rest], q[rest]), bits
