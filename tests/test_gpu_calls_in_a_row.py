"""Calls of the operators around the layer one after another without a wait between them:
a kernel may be on the GPU before the one ahead of it has finished (programmatic launch),
so what it reads of that one's outputs must be what was written last.  The results are
compared bit for bit with the same calls made one at a time.
"""
from __future__ import annotations

import pytest
import torch

import sparse_mixture_experts_argmax_b200 as swl
from sparse_mixture_experts_argmax_b200 import build as swl_build

pytestmark = pytest.mark.gpu

F, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    swl_build.build()
    swl.lib()


def _n(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _offsets(sizes):
    return torch.tensor([sum(sizes[:i]) for i in range(len(sizes) + 1)], dtype=torch.int32,
                        device="cuda")


@pytest.mark.parametrize("dtype", [F, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows", [8, 400])
def test_other_offsets_on_the_same_workspace(rows, dtype):
    """Groups that change from call to call, forward and backward, on one workspace."""
    N, K, O = 6, 136, 264
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, dy = _n(g, (rows, K), dtype), _n(g, (rows, O), dtype)
    W, b = _n(g, (N, O, K), dtype, K ** -0.5), _n(g, (N, O), dtype)
    q = rows // 8
    offs = [_offsets(s) for s in ([8 * q, 0, 0, 0, 0, 0], [0, 0, 0, 0, 0, 8 * q], [q, q, q, q, q, 3 * q],
                                  [0, 5 * q, 0, 3 * q, 0, 0], [3 * q, 0, 0, 0, 5 * q, 0])]
    n = swl.switch_layer_grouped_workspace_size(rows, K, O, N, swl.dtype_code(dtype))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def call(off, out):
        swl.grouped_matmul(x, off, W, bias=b, out=out["y"], workspace=ws, check=False)
        swl.grouped_matmul_backward(dy, x, off, W, dx=out["dx"], dW=out["dW"], db=out["db"],
                                    workspace=ws, check=False)

    def outs():
        return [dict(y=torch.zeros_like(dy), dx=torch.zeros_like(x), dW=torch.zeros_like(W),
                     db=torch.zeros_like(b)) for _ in offs]

    want = outs()
    for off, o in zip(offs, want):
        call(off, o)
        torch.cuda.synchronize()
        assert swl.lib().switch_layer_device_status(ws.data_ptr(), None) == 0

    def same(got):
        for i, (a, c) in enumerate(zip(got, want)):
            for k in a:
                assert torch.equal(a[k], c[k]), (i, k)

    for _ in range(20):
        got = outs()
        for off, o in zip(offs, got):
            call(off, o)
        same(got)
    got = outs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for off, o in zip(offs, got):
            call(off, o)
    for _ in range(20):
        for o in got:
            for t in o.values():
                t.zero_()
        graph.replay()
        same(got)


@pytest.mark.parametrize("dtype", [F, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows", [5, 300])
def test_each_call_reads_what_the_last_one_wrote(rows, dtype):
    """A chain of products through two buffers that take turns."""
    N, K, steps = 3, 256, 40
    g = torch.Generator(device="cuda").manual_seed(rows + 1)
    start = _n(g, (rows, K), dtype)
    W = _n(g, (N, K, K), dtype, K ** -0.5)
    off = _offsets([rows - 4, 0, 4])
    n = swl.switch_layer_grouped_workspace_size(rows, K, K, N, swl.dtype_code(dtype))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    bufs = [torch.empty_like(start), torch.empty_like(start)]

    def chain(wait):
        bufs[0].copy_(start)
        for i in range(steps):
            swl.grouped_matmul(bufs[i & 1], off, W, out=bufs[1 - (i & 1)], workspace=ws, check=False)
            if wait:
                torch.cuda.synchronize()

    chain(True)
    want = bufs[0].clone()
    assert torch.isfinite(want).all() and want.count_nonzero() > 0
    for _ in range(10):
        chain(False)
        assert torch.equal(bufs[0], want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(False)
    for _ in range(10):
        bufs[0].zero_()
        graph.replay()
        assert torch.equal(bufs[0], want)


@pytest.mark.parametrize("dtype", [F, BF], ids=["f32", "bf16"])
def test_products_behind_a_norm_that_sums_no_columns(dtype):
    """The backward pass of a residual with a gate alone has one kernel; the product behind it
    reads its dy."""
    T, d, N = 200, 131 if dtype == F else 136, 3
    g = torch.Generator(device="cuda").manual_seed(9)
    dr, y = _n(g, (T, d), dtype), _n(g, (T, d), dtype)
    gate = torch.rand(T, generator=g, device="cuda")
    W = _n(g, (N, d, d), dtype, d ** -0.5)
    off = _offsets([70, 0, 130])
    want = swl.norm_residual_backward(dr, None, y, y=y, gate=gate)["dy"]
    torch.cuda.synchronize()
    product = swl.grouped_matmul(want, off, W)
    for _ in range(20):
        dy = swl.norm_residual_backward(dr, None, y, y=y, gate=gate)["dy"]
        got = swl.grouped_matmul(dy, off, W, out=torch.zeros_like(product), check=False)
        assert torch.equal(dy, want) and torch.equal(got, product)


def test_a_workspace_for_the_largest_batch_serves_smaller_ones():
    N, K, O = 16, 64, 136
    g = torch.Generator(device="cuda").manual_seed(12)
    x, dy = _n(g, (40 * N, K), BF), _n(g, (40 * N, O), BF)
    W = _n(g, (N, O, K), BF, K ** -0.5)
    ws = torch.empty(swl.switch_layer_grouped_workspace_size(40 * N, K, O, N, swl.SWL_BF16),
                     dtype=torch.uint8, device="cuda")
    for rows in (40 * N, 40 * N - 1, 39 * N, 100, 1):
        off = _offsets([rows // 2] + [0] * (N - 2) + [rows - rows // 2])
        args = dy[:rows], x[:rows], off, W
        got = swl.grouped_matmul_backward(*args, workspace=ws)
        want = swl.grouped_matmul_backward(*args)
        for k in want:
            assert torch.equal(got[k], want[k]), (rows, k)
        assert torch.equal(swl.grouped_matmul(x[:rows], off, W, workspace=ws),
                           swl.grouped_matmul(x[:rows], off, W))


def test_streams_given_as_handles():
    """0 and 1 are the legacy default stream's handles, 2 the calling thread's default stream."""
    g = torch.Generator(device="cuda").manual_seed(13)
    x, W, off = _n(g, (40, 64), F), _n(g, (2, 24, 64), F), _offsets([10, 30])
    w = torch.ones(64, device="cuda")
    want = swl.grouped_matmul(x, off, W)
    wantg = swl.grouped_matmul_backward(want, x, off, W)
    norm = swl.norm_residual(x, w_pre=w)
    back = swl.norm_residual_backward(None, x, x, w_pre=w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for handle in (0, 1, 2, side.cuda_stream):
        y = swl.grouped_matmul(x, off, W, stream=handle)
        gr = swl.grouped_matmul_backward(want, x, off, W, stream=handle)
        nr = swl.norm_residual(x, w_pre=w, stream=handle)
        nb = swl.norm_residual_backward(None, x, x, w_pre=w, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(nr["h"], norm["h"]), handle
        assert all(torch.equal(gr[k], wantg[k]) for k in wantg), handle
        assert torch.equal(nb["dx"], back["dx"]) and torch.equal(nb["dw_pre"], back["dw_pre"]), handle
