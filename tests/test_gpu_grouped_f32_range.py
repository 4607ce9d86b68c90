"""Grouped products of fp32 tensors at the ends of the range, by the three-piece split (more
than 32 rows, and the backward pass at any) and by plain fp32 sums (up to 32 rows).

Tolerance: (n + 6) 2^-23 S for a sum of n products of absolute size S, as for ordinary
numbers (what the split leaves out, 2^-28, is inside); a number's pieces end at 2^-133, the
smallest bf16, so each factor may be off by that, times the other one; every one of the
eight products, and the result, may be off by the smallest fp32 number, 2^-149.
"""
from __future__ import annotations

import pytest
import torch

import sparse_mixture_experts_argmax_b200 as swl
from sparse_mixture_experts_argmax_b200 import build as swl_build

pytestmark = pytest.mark.gpu

F = torch.float32
BIG = torch.finfo(F).max
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    swl_build.build()
    swl.lib()


def _numbers(seed, shape, exponent):
    """Random signs and mantissas of 24 bits (fewer below 2^-126), one binary exponent."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    m = 1 + torch.rand(shape, generator=g, device="cuda", dtype=torch.float64)
    sign = 2.0 * torch.randint(0, 2, shape, generator=g, device="cuda") - 1
    return (sign * m * 2.0 ** exponent).float()


def _offsets(rows):
    return torch.tensor([0, rows], dtype=torch.int32, device="cuda")


def _close(got, a, b, what):
    """got against a @ b in 64 bits."""
    a, b = a.double(), b.double()
    n = a.shape[1]
    want, size = a @ b, a.abs() @ b.abs()
    tol = ((n + 6) * 2.0 ** -23 * size + 2.0 ** -24 * want.abs() + (8 * n + 1) * 2.0 ** -149 +
           2.0 ** -133 * (a.abs().sum(1, keepdim=True) + b.abs().sum(0, keepdim=True)))
    diff = (got.double() - want).abs()
    assert (diff <= tol).all(), (what, float((diff / tol).max()))


# aligned rows of 16 bytes, of 8 bytes, and of neither
@pytest.mark.parametrize("K,O", [(64, 72), (70, 66), (63, 41)])
@pytest.mark.parametrize("small,large", [(-109, 100), (-111, 100), (-113, 100), (-120, 110), (-126, 110),
                                         (-130, 120), (-140, 120), (-70, -60), (-100, -45), (30, 90)])
@pytest.mark.parametrize("rows", [20, 40])
def test_tiny_numbers_beside_large_ones(rows, small, large, K, O):
    off = _offsets(rows)
    x, W, dy = _numbers(1, (rows, K), small), _numbers(2, (1, O, K), large), _numbers(3, (rows, O), small)
    _close(swl.grouped_matmul(x, off, W), x, W[0].T, "y")
    x = _numbers(4, (rows, K), large)
    g = swl.grouped_matmul_backward(dy, x, off, W)
    _close(g["dx"], dy, W[0], "dx")
    _close(g["dW"][0], dy.T, x, "dW")


@pytest.mark.parametrize("K", [64, 70, 63])
@pytest.mark.parametrize("rows", [20, 32, 33, 40])
def test_the_ends_of_the_range(rows, K):
    """One product a sum, so that the result is the factor itself or half of it: the largest
    numbers (whose leading piece must not round to infinity), the smallest, 0, inf, NaN."""
    off = _offsets(rows)
    special = {4: BIG, 5: INF, 6: NAN, 7: -BIG, 8: 2.0 ** -110, 9: -2.0 ** -126, 10: -INF, 11: 0.0}
    v = torch.linspace(1, 2, rows, device="cuda")
    for r, s in special.items():
        v[r] = s
    x = torch.zeros((rows, K), device="cuda")
    x[:, 3] = v
    W = torch.zeros((1, 8, K), device="cuda")
    W[0, :, 3] = 1.0
    W[0, 1, 3] = -0.5
    dy = torch.zeros((rows, 8), device="cuda")
    dy[:, 5] = v
    Wb = torch.zeros((1, 8, K), device="cuda")
    Wb[0, 5] = 1.0
    Wb[0, 5, 1] = -0.5
    y = swl.grouped_matmul(x, off, W)
    g = swl.grouped_matmul_backward(dy, x * 0, off, Wb)
    for r in range(rows):
        want = float(v[r])
        for got in (y[r], g["dx"][r]):
            if want != want:
                assert got.isnan().all(), r
            elif abs(want) == INF:
                # up to 32 rows of y are fp32 sums, with their infinities; the split's pieces of
                # the other factor, some of them zero, make NaN of one
                plain = got.data_ptr() == y[r].data_ptr() and rows <= 32
                assert got[0] == want and got[1] == -want if plain else got.isnan().all(), r
            else:
                assert float(got[0]) == want and float(got[1]) == -0.5 * want, (r, got[:2], want)


@pytest.mark.parametrize("value", [INF, -INF, NAN], ids=str)
def test_what_is_not_finite_stays_in_its_group_and_row(value):
    K, O = 66, 41
    off = torch.tensor([0, 40, 90, 90, 150], dtype=torch.int32, device="cuda")
    x, dy, W = _numbers(5, (150, K), 0), _numbers(6, (150, O), 0), _numbers(7, (4, O, K), -3)
    y, g = swl.grouped_matmul(x, off, W), swl.grouped_matmul_backward(dy, x, off, W)
    x1, dy1 = x.clone(), dy.clone()
    x1[60, 7] = value
    dy1[100, 11] = value
    y1, g1 = swl.grouped_matmul(x1, off, W), swl.grouped_matmul_backward(dy1, x1, off, W)
    row = torch.arange(150, device="cuda")
    assert torch.equal(y1[row != 60], y[row != 60]) and not torch.isfinite(y1[60]).any()
    assert torch.equal(g1["dx"][row != 100], g["dx"][row != 100]) and not torch.isfinite(g1["dx"][100]).any()
    for e in (0, 2):
        assert torch.equal(g1["dW"][e], g["dW"][e])
    assert not torch.isfinite(g1["dW"][1][:, 7]).any() and not torch.isfinite(g1["dW"][3][11]).any()
    keep = torch.arange(K, device="cuda") != 7
    assert torch.equal(g1["dW"][1][:, keep], g["dW"][1][:, keep])
    keep = torch.arange(O, device="cuda") != 11
    assert torch.equal(g1["dW"][3][keep], g["dW"][3][keep])
