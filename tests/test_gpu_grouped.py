"""switch_layer_grouped_matmul and its backward pass against the products in 64 bits.

Tolerance: a sum of n products of exact factors in fp32, every partial sum off by at
most 2^-23 of the sum S of the absolute products (rounded or truncated), is off by at
most (n + 2) 2^-23 S; then half a step of the output type.  The products that stand
for one of two fp32 numbers leave out under 2^-28 of it.
"""
from __future__ import annotations

import pytest
import torch

import sparse_mixture_experts_argmax_b200 as swl
from sparse_mixture_experts_argmax_b200 import build as swl_build

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    swl_build.build()
    swl.lib()


def _case(sizes, K, O, dtype, before=0, after=0, bias=True, seed=0):
    """Rows before the first group and behind the last hold NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    N, M = len(sizes), sum(sizes)
    R = before + M + after
    off = torch.tensor([before] + [before + sum(sizes[:i + 1]) for i in range(N)] if N < 100 else
                       (before + torch.tensor([0] + list(sizes)).cumsum(0)).tolist(),
                       dtype=torch.int32, device="cuda")
    c = dict(x=n(R, K), W=n(N, O, K, std=K ** -0.5), bias=n(N, O) if bias else None,
             dy=n(R, O), offsets=off, sizes=list(sizes), before=before)
    for t in ("x", "dy"):
        c[t][:before] = float("nan")
        c[t][R - after:] = float("nan")
    return c


def _close(got, want, size, terms, what):
    tol = (terms + 6) * 2.0 ** -23 * size + HALF[got.dtype] * want.abs() + 1e-38
    diff = (got.double() - want).abs()
    assert (diff <= tol).all(), (what, float((diff / tol).nan_to_num(1e30).max()))


def _check(c, fwd=True, bwd=True):
    x, W, dy, off = c["x"], c["W"], c["dy"], c["offsets"].tolist()
    N, O, K = W.shape
    R = x.shape[0]
    dt = x.dtype
    mark = 7.0
    if fwd:
        out = torch.full((R, O), mark, dtype=dt, device="cuda")
        assert swl.grouped_matmul(x, c["offsets"], W, bias=c["bias"], out=out) is out
    if bwd:
        dx = torch.full((R, K), mark, dtype=dt, device="cuda")
        dW = torch.full((N, O, K), mark, dtype=dt, device="cuda")
        db = torch.full((N, O), mark, dtype=dt, device="cuda")
        swl.grouped_matmul_backward(dy, x, c["offsets"], W, dx=dx, dW=dW, db=db)
    outside = torch.ones(R, dtype=torch.bool, device="cuda")
    outside[off[0]:off[-1]] = False
    if fwd:
        assert (out[outside] == mark).all()
    if bwd:
        assert (dx[outside] == mark).all()
    for e in range(N):
        a, b = off[e], off[e + 1]
        X, Wd, G = x[a:b].double(), W[e].double(), dy[a:b].double()
        if fwd and b > a:
            y, s = X @ Wd.T, X.abs() @ Wd.abs().T
            if c["bias"] is not None:
                y, s = y + c["bias"][e].double(), s + c["bias"][e].double().abs()
            _close(out[a:b], y, s, K, ("y", e))
        if bwd:
            if b > a:
                _close(dx[a:b], G @ Wd, G.abs() @ Wd.abs(), O, ("dx", e))
            _close(dW[e], G.T @ X, G.abs().T @ X.abs(), b - a, ("dW", e))
            _close(db[e], G.sum(0), G.abs().sum(0), b - a, ("db", e))


EDGES = [1, 2, 15, 16, 17, 31, 32, 33, 0, 63, 64, 65, 127, 128, 129, 0, 255, 256, 257, 300]


@pytest.mark.parametrize("K,O", [(8, 8), (24, 40), (64, 64), (72, 136), (128, 256), (264, 520), (1032, 16)])
def test_bf16_edges(K, O):
    _check(_case(EDGES, K, O, BF, before=3, after=5))
    _check(_case([5], K, O, BF, bias=False))
    _check(_case([0, 0, 1, 0], K, O, BF, after=1))


@pytest.mark.parametrize("K,O", [(1, 1), (3, 5), (17, 33), (64, 64), (129, 257), (765, 100), (40, 1021)])
def test_f32_edges(K, O):
    _check(_case(EDGES, K, O, F, before=3, after=5))
    _check(_case([5], K, O, F, bias=False))
    _check(_case([0, 0, 1, 0], K, O, F, after=1))


@pytest.mark.parametrize("dtype", [F, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 16, 17, 40])
def test_few_rows_over_many_groups(rows, dtype):
    """Decoded tokens: a handful of rows, spread or all in one group."""
    g = torch.Generator().manual_seed(rows)
    for N, spread in ((1, False), (64, True), (64, False), (1500, True)):
        sizes = [0] * N
        for _ in range(rows):
            sizes[int(torch.randint(N, (1,), generator=g)) if spread else N // 2] += 1
        K, O = (136, 72) if N == 1500 else (1024, 520)
        _check(_case(sizes, K, O, dtype, before=rows % 3, after=rows % 2), bwd=N < 1500)


@pytest.mark.parametrize("dtype,K,O", [(BF, 768, 1024), (F, 256, 300)], ids=["bf16", "f32"])
@pytest.mark.parametrize("sizes", [[2000], [700, 0, 1, 90, 1500, 64], [40] * 64, [1300, 1300]],
                         ids=["one", "ragged", "even", "two"])
def test_larger(sizes, dtype, K, O):
    _check(_case(sizes, K, O, dtype, after=100))


def test_long_sums():
    _check(_case([64, 9000, 3], 64, 128, BF, bias=False))
    _check(_case([64, 5000, 3], 64, 100, F, bias=False))
    _check(_case([30, 50], 8200, 64, BF))


@pytest.mark.parametrize("dtype", [F, BF], ids=["f32", "bf16"])
def test_one_output_at_a_time_and_empty_batch(dtype):
    c = _case([33, 0, 70], 64, 96, dtype, after=2)
    full = swl.grouped_matmul_backward(c["dy"], c["x"], c["offsets"], c["W"])
    for k, like in (("dx", c["x"]), ("dW", c["W"]), ("db", c["bias"])):
        got = swl.grouped_matmul_backward(c["dy"], c["x"], c["offsets"], c["W"],
                                          **{k: torch.zeros_like(like)})
        assert torch.equal(got[k], full[k]), k
        assert [q for q in got if got[q] is not None] == [k]
    y = swl.grouped_matmul(c["x"], c["offsets"], c["W"])
    assert (y[-2:] == 0).all()                    # allocated here: rows of no group are zero
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    none = c["x"][:0], c["dy"][:0]
    assert swl.grouped_matmul(none[0], off, c["W"]).shape == (0, 96)
    g = swl.grouped_matmul_backward(none[1], none[0], off, c["W"])
    assert g["dx"].shape == (0, 64) and (g["dW"] == 0).all() and (g["db"] == 0).all()


@pytest.mark.parametrize("dtype", [F, BF], ids=["f32", "bf16"])
def test_non_finite_rows_stay_in_their_group(dtype):
    sizes = [20, 45, 70, 9]
    c = _case(sizes, 64, 136, dtype)
    off = c["offsets"].tolist()
    clean = swl.grouped_matmul_backward(c["dy"], c["x"], c["offsets"], c["W"])
    y = swl.grouped_matmul(c["x"], c["offsets"], c["W"], bias=c["bias"])
    c["x"][off[1] + 3] = float("nan")
    c["dy"][off[2] - 1] = float("inf")             # the last row of group 1
    y1 = swl.grouped_matmul(c["x"], c["offsets"], c["W"], bias=c["bias"])
    row = torch.arange(y.shape[0], device="cuda")
    assert torch.equal(y1[row != off[1] + 3], y[row != off[1] + 3])
    assert y1[off[1] + 3].isnan().all()
    g = swl.grouped_matmul_backward(c["dy"], c["x"], c["offsets"], c["W"])
    assert torch.equal(g["dx"][row != off[2] - 1], clean["dx"][row != off[2] - 1])
    for e in (0, 2, 3):
        assert torch.equal(g["dW"][e], clean["dW"][e]) and torch.equal(g["db"][e], clean["db"][e])
    assert not torch.isfinite(g["dW"][1]).any()


@pytest.mark.parametrize("dtype", [F, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("bad", [[0, 10, 5, 20], [-1, 5, 10, 20], [0, 5, 10, 41], [0, 1 << 30, 3, 4]],
                         ids=["falling", "negative", "beyond", "huge"])
@pytest.mark.parametrize("rows", [40, 8])
def test_bad_offsets_are_refused_on_the_device(rows, bad, dtype):
    bad = torch.tensor([min(b, rows + 1) if b == 41 else b for b in bad], dtype=torch.int32,
                       device="cuda")
    x, dy = torch.ones((rows, 64), dtype=dtype, device="cuda"), torch.ones((rows, 72), dtype=dtype, device="cuda")
    W = torch.ones((3, 72, 64), dtype=dtype, device="cuda")
    outs = dict(dx=torch.full_like(x, 7), dW=torch.full_like(W, 7), db=torch.full_like(W[:, :, 0], 7))
    y = torch.full_like(dy, 7)
    with pytest.raises(swl.SwitchLayerError) as e:
        swl.grouped_matmul(x, bad, W, out=y)
    assert e.value.status == 5
    with pytest.raises(swl.SwitchLayerError) as e:
        swl.grouped_matmul_backward(dy, x, bad, W, **outs)
    assert e.value.status == 5
    assert (y == 7).all() and all((t == 7).all() for t in outs.values())
    good = torch.tensor([0, 1, 5, 8], dtype=torch.int32, device="cuda")
    ws = torch.empty(swl.switch_layer_grouped_workspace_size(rows, 64, 72, 3, swl.dtype_code(dtype)),
                     dtype=torch.uint8, device="cuda")
    with pytest.raises(swl.SwitchLayerError):
        swl.grouped_matmul(x, bad, W, out=y, workspace=ws)
    swl.grouped_matmul(x, good, W, out=y, workspace=ws)      # the next call starts afresh
    assert (y[:8] == 64).all() and (y[8:] == 7).all()


@pytest.mark.parametrize("dtype", [F, BF], ids=["f32", "bf16"])
def test_capture_streams_and_repeats(dtype):
    c = _case([100, 0, 37, 290], 128, 200, dtype, after=9)
    args = c["dy"], c["x"], c["offsets"], c["W"]
    want = swl.grouped_matmul(c["x"], c["offsets"], c["W"], bias=c["bias"])
    wantg = swl.grouped_matmul_backward(*args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = swl.grouped_matmul(c["x"], c["offsets"], c["W"], bias=c["bias"], check=False)
        g = swl.grouped_matmul_backward(*args, check=False)
    for _ in range(3):
        graph.replay()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:                    # two calls at once, a workspace each
        s.wait_stream(torch.cuda.current_stream())
        got.append((swl.grouped_matmul(c["x"], c["offsets"], c["W"], bias=c["bias"], stream=s, check=False),
                    swl.grouped_matmul_backward(*args, stream=s, check=False)))
    torch.cuda.synchronize()
    for yy, gg in got + [(y, g)]:
        assert torch.equal(yy, want)
        for k in wantg:
            assert torch.equal(gg[k], wantg[k]), k
    # new offsets under the same graph
    other = _case([0, 300, 100, 27], 128, 200, dtype, after=9)
    c["offsets"].copy_(other["offsets"])
    graph.replay()
    again = swl.grouped_matmul_backward(*args)
    for k in ("dW", "db"):
        assert torch.equal(g[k], again[k]), k


def test_gradients_against_differences():
    """dW, dx and db are the slopes of the forward pass (linear in each: the
    difference quotient is exact up to fp32 sums of 30 terms, 1e-4)."""
    c = _case([3, 0, 5], 6, 7, F)
    got = swl.grouped_matmul_backward(c["dy"], c["x"], c["offsets"], c["W"])

    def loss(x, W, b):
        return float((swl.grouped_matmul(x, c["offsets"], W, bias=b).double() * c["dy"].double()).sum())

    for name, i in (("x", 0), ("W", 1), ("bias", 2)):
        t = [c["x"], c["W"], c["bias"]]
        g = got[{"x": "dx", "W": "dW", "bias": "db"}[name]].view(-1)
        for at in range(0, t[i].numel(), 5):
            up, down = t[i].clone(), t[i].clone()
            up.view(-1)[at] += 0.5
            down.view(-1)[at] -= 0.5
            slope = loss(*(t[:i] + [up] + t[i + 1:])) - loss(*(t[:i] + [down] + t[i + 1:]))
            assert abs(slope - float(g[at])) <= 1e-4 * (1 + abs(slope)), (name, at)


def test_wrapper_refusals():
    c = _case([3, 4], 16, 24, BF)
    x, W, off = c["x"], c["W"], c["offsets"]
    for args, err in (((x[:, :8], off, W), ValueError), ((x.float(), off, W), TypeError),
                      ((x, off.long(), W), TypeError), ((x, off[:2], W), ValueError),
                      ((x, off.cpu(), W), ValueError), ((x[0], off, W), ValueError),
                      ((x, off, W[:, :, :8].contiguous()), ValueError),
                      ((x[:, :12].contiguous(), off, W[:, :, :12].contiguous()), swl.SwitchLayerError)):
        with pytest.raises(err):
            swl.grouped_matmul(*args)
    with pytest.raises(ValueError):
        swl.grouped_matmul(x, off, W, out=torch.zeros((6, 24), dtype=BF, device="cuda"))
    with pytest.raises(swl.SwitchLayerError):
        swl.grouped_matmul(x, off, W, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    square = torch.zeros((2, 16, 16), dtype=BF, device="cuda")
    with pytest.raises(swl.SwitchLayerError):
        swl.grouped_matmul(x, off, square, out=x)             # in place


def test_f32_values_at_the_ends_of_the_range():
    """The largest numbers (whose leading piece must not round to infinity), tiny ones,
    infinities and NaN, by rows that start on 16-byte boundaries and by rows that do not."""
    big = torch.finfo(F).max
    for K in (64, 63):
        x = torch.zeros((20, K), device="cuda")
        W = torch.zeros((1, 8, K), device="cuda")
        W[0, :, 3] = 1.0
        W[0, 1, 3] = -0.5
        x[:, 3] = torch.linspace(1, 2, 20, device="cuda")
        x[4, 3], x[5, 3], x[6, 3] = big, float("inf"), float("nan")
        x[7, 3], x[8, 3] = -big, 2.0 ** -100
        off = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
        y = swl.grouped_matmul(x, off, W)
        for r in range(20):
            want = x[r, 3]
            if r == 5:
                # not finite, as documented.  By arithmetic it is NaN: W = 1 is the pieces
                # 1, 0, 0, and among the products infinity meets the zeros
                assert not torch.isfinite(y[r]).any()
            elif r == 6:
                assert y[r].isnan().all()
            else:
                assert abs(float(y[r, 0]) - float(want)) <= 2.0 ** -22 * abs(float(want))
                assert abs(float(y[r, 1]) + 0.5 * float(want)) <= 2.0 ** -22 * abs(float(want))
