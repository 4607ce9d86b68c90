"""Two host threads that call the library at the same time, each on a stream and a
workspace of its own, with shapes whose kernels take different amounts of shared memory."""
from __future__ import annotations

import threading

import pytest
import torch

import sparse_mixture_experts_argmax_b200 as swl
from sparse_mixture_experts_argmax_b200 import build as swl_build

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    swl_build.build()
    swl.lib()


def _at_once(jobs, calls):
    """Each job `calls` times in a thread of its own; the errors that came up."""
    errors, ready = [], threading.Barrier(len(jobs))

    def body(job):
        try:
            ready.wait()
            for _ in range(calls):
                job()
        except Exception as e:  # noqa: BLE001 - reported below
            errors.append(repr(e))

    threads = [threading.Thread(target=body, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return errors


def _n(seed, shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)


def _layer(seed, T, d, d_ff, N, cf):
    inputs = {"x": _n(seed, (T, d)), "W_r": _n(seed + 1, (N, d), d ** -0.5).float(), "b_r": None,
              "W1": _n(seed + 2, (N, d_ff, d), d ** -0.5), "b1": _n(seed + 3, (N, d_ff), 0.1),
              "W2": _n(seed + 4, (N, d, d_ff), d_ff ** -0.5), "b2": _n(seed + 5, (N, d), 0.1)}
    ws = swl.alloc_workspace(T, d, d_ff, N, BF, cf)
    stream = torch.cuda.Stream()
    got = {}

    def job():
        with torch.cuda.stream(stream):
            got["out"] = swl.forward(inputs, cf, workspace=ws, check=False)["out"]
    return job, got


def _products(seed, sizes, K, O, backward):
    """A product of one direction on a stream of its own; its outputs are returned as well."""
    N, R = len(sizes), sum(sizes)
    x, dy, W = _n(seed, (R, K)), _n(seed + 1, (R, O)), _n(seed + 2, (N, O, K), K ** -0.5)
    off = torch.tensor([sum(sizes[:i]) for i in range(N + 1)], dtype=torch.int32, device="cuda")
    ws = torch.empty(swl.switch_layer_grouped_workspace_size(R, K, O, N, swl.SWL_BF16),
                     dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(W if backward else dy)
    stream = torch.cuda.Stream()

    def job():
        if backward:
            swl.grouped_matmul_backward(dy, x, off, W, dW=out, workspace=ws, stream=stream, check=False)
        else:
            swl.grouped_matmul(x, off, W, out=out, workspace=ws, stream=stream, check=False)
    return job, out, ws


def _in_a_new_thread(job):
    """A thread whose first call of the CUDA runtime or driver is the library's."""
    return _at_once([job], 1)


def test_first_call_of_a_thread():
    for backward in (False, True):
        job, out, _ = _products(40, [20, 30], 64, 64, backward)
        torch.cuda.synchronize()
        assert _in_a_new_thread(job) == [], backward
        got = out.clone()
        job()
        torch.cuda.synchronize()
        assert torch.equal(out, got) and got.count_nonzero() > 0
    for shape in ((300, 64, 64, 6, 1.25), (512, 64, 64, 600, 1.0)):
        job, got = _layer(50, *shape)
        torch.cuda.synchronize()
        assert _in_a_new_thread(job) == [], shape
        first = got["out"].clone()
        job()
        torch.cuda.synchronize()
        assert torch.equal(got["out"], first)


@pytest.mark.parametrize("backward", [False, True], ids=["y", "dW"])
def test_grouped_products_of_different_shapes(backward):
    torch.cuda.synchronize()
    # tiles of 64 and of 256 rows; dW with narrow and with wide columns
    jobs = [_products(10 * i, *((([20] * 4, 64, 64) if i % 2 else ([250, 60], 256, 64))), backward)
            for i in range(6)]
    torch.cuda.synchronize()
    want = []
    for job, out, _ in jobs:
        job()
        torch.cuda.synchronize()
        want.append(out.clone())
    assert _at_once([j for j, _, _ in jobs], 4000) == []
    for (_, out, ws), w in zip(jobs, want):
        assert swl.lib().switch_layer_device_status(ws.data_ptr(), None) == 0
        assert torch.equal(out, w)


def test_layers_of_different_shapes():
    """A many-expert layer (streaming softmax), a small one (fused router of two stages) and
    one of few tokens."""
    jobs = [_layer(1, 512, 64, 64, 600, 1.0), _layer(11, 40000, 64, 64, 8, 1.25),
            _layer(21, 300, 128, 128, 6, 1.25), _layer(31, 256, 64, 64, 1600, 1.0)]
    torch.cuda.synchronize()
    want = []
    for job, got in jobs:
        job()
        torch.cuda.synchronize()
        want.append(got["out"].clone())
    assert _at_once([j for j, _ in jobs], 400) == []
    for (_, got), w in zip(jobs, want):
        assert torch.equal(got["out"], w)
