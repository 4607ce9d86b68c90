"""Grouped products of very long sums: a single tile may take longer than the limit of a wait
inside the kernels, which must then grow with the sum; and sums of positive terms must not
come out short, although the tensor cores cut their running sums instead of rounding them."""
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


def _uniform(seed, shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(shape, generator=g, device="cuda").to(dtype)


def _not_short(got, a, b, what):
    """got against a @ b, positive terms.  The unrounded sum s is off by `cut` of it at most: a
    piece of 32768 terms is cut 2048 times (16 terms at once, their products aligned with
    2^-23 of the running sum and the sum cut to 2^-23), and every piece's sum is rounded.  got
    is s rounded, so |got - s| <= |R - s| for the exact sum's own rounding R, and
    |got - want| <= |R - s| + |s - want| <= |R - want| + 2 |s - want|.  (Sums of so many
    terms are nearly equal, and round alike: their errors do not average out.)"""
    want = a.double() @ b.double()
    pieces = -(-a.shape[1] // 32768)
    cut = (2 * 2048 + pieces) * 2.0 ** -23
    over = ((got.double() - want).abs() - (want.to(got.dtype).double() - want).abs()) / want
    assert float(over.max()) <= 2 * cut, (what, float(over.max()))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows", [1 << 16, 1 << 20, (1 << 21) + 12345])
def test_weight_gradients_of_many_rows_are_not_short(rows, dtype):
    x, dy = _uniform(1, (rows, 72), dtype), _uniform(2, (rows, 136), dtype)
    W = torch.zeros((1, 136, 72), dtype=dtype, device="cuda")
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    g = swl.grouped_matmul_backward(dy, x, off, W)
    _not_short(g["dW"][0], dy.T, x, "dW")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_wide_rows_are_not_short(dtype):
    rows, wide = 70, (1 << 18) + 8
    off = torch.tensor([0, 50, rows], dtype=torch.int32, device="cuda")
    x, W = _uniform(3, (rows, wide), dtype), _uniform(4, (2, 40, wide), dtype)
    b = _uniform(5, (2, 40), dtype)
    y = swl.grouped_matmul(x, off, W, bias=b)
    dx = swl.grouped_matmul_backward(x, y[:, :8].contiguous(), off, W.transpose(1, 2)[:, :, :8].contiguous(),
                                     dx=torch.zeros_like(y[:, :8].contiguous()))["dx"]
    for e, r in ((0, slice(0, 50)), (1, slice(50, rows))):
        # the bias, under 2^-16 of the sums, as one term more
        one = torch.ones((x[r].shape[0], 1), dtype=dtype, device="cuda")
        _not_short(y[r], torch.cat([x[r], one], 1), torch.cat([W[e].T, b[e][None]]), ("y", e))
        _not_short(dx[r], x[r], W[e].T[:, :8], ("dx", e))


def test_pieces_of_many_groups_and_tiles():
    """Groups around whole pieces among small and empty ones, several tiles per group, repeated
    and captured: equal bit for bit, and right."""
    sizes = [5, 32768, 0, 32769, 40000, 64, 65536, 65537, 1]
    K, O = 520, 264
    off = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(6)
    R = sum(sizes)
    x = torch.randn((R, K), generator=g, device="cuda").bfloat16()
    dy = torch.randn((R, O), generator=g, device="cuda").bfloat16()
    W = torch.zeros((len(sizes), O, K), dtype=torch.bfloat16, device="cuda")
    dW = torch.full_like(W, 7)
    swl.grouped_matmul_backward(dy, x, off, W, dW=dW)
    at = off.tolist()
    for e in range(len(sizes)):
        G, X = dy[at[e]:at[e + 1]].double(), x[at[e]:at[e + 1]].double()
        want, size = G.T @ X, G.abs().T @ X.abs()
        tol = (min(sizes[e], 32768) + 8) * 2.0 ** -23 * size + 2.0 ** -8 * want.abs()
        assert ((dW[e].double() - want).abs() <= tol).all(), e
    again = torch.zeros_like(W)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        swl.grouped_matmul_backward(dy, x, off, W, dW=again, check=False)
    for _ in range(3):
        again.zero_()
        graph.replay()
        assert torch.equal(again, dW)
