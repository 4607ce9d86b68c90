"""Grouped products whose sums are so long that a single tile takes longer than the limit of
a wait inside the kernels, which must then grow with the sum."""
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


@pytest.fixture
def one_ms():
    swl.switch_layer_set_wait_limit_ns(1_000_000)
    yield
    swl.switch_layer_set_wait_limit_ns(0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_sums_longer_than_a_wait(one_ms, dtype):
    """2^22 terms, whole numbers: every partial sum is exact in fp32 (and 2^22 in bf16)."""
    n, w = 1 << 22, 8
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    x = torch.ones((n, w), dtype=dtype, device="cuda")
    dy = torch.ones((n, w), dtype=dtype, device="cuda")
    W = torch.ones((1, w, w), dtype=dtype, device="cuda")
    g = swl.grouped_matmul_backward(dy, x, off, W)
    assert (g["dW"] == n).all() and (g["db"] == n).all() and (g["dx"] == w).all()
    rows = 40                                     # too many for the few-row kernel
    x = torch.ones((rows, n), dtype=dtype, device="cuda")
    W = torch.ones((1, w, n), dtype=dtype, device="cuda")
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    assert (swl.grouped_matmul(x, off, W) == n).all()
