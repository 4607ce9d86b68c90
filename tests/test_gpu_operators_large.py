"""The operators around the layer on buffers whose element offsets pass 2^31, on very many
groups, and at addresses that only the element's own size divides."""
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


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _n(seed, shape, dtype, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype) * std


def _close(got, want, size, terms):
    half = 2.0 ** -8 if got.dtype == BF else 2.0 ** -24
    tol = (terms + 6) * 2.0 ** -23 * size + half * want.abs() + 1e-38
    assert ((got.double() - want).abs() <= tol).all()


def _product(got, a, b):
    a, b = a.double(), b.double()
    _close(got, a @ b, a.abs() @ b.abs(), a.shape[1])


@pytest.mark.parametrize("dtype", [F, BF], ids=["f32", "bf16"])
def test_rows_past_32_bits(dtype):
    """y has 2^31 elements and some rows more; the last group lies behind them."""
    K, O = 16, 4096
    R = (1 << 31) // O + 700
    x, dy, W = _n(1, (R, K), dtype), _n(2, (R, O), dtype, 0.1), _n(3, (3, O, K), dtype)
    cut = R - 333
    off = torch.tensor([5, 5, cut, R], dtype=torch.int32, device="cuda")
    y = swl.grouped_matmul(x, off, W)
    assert (y[:5] == 0).all()
    for rows, e in ((slice(5, 105), 1), (slice(cut - 50, cut), 1), (slice(cut, R), 2)):
        _product(y[rows], x[rows], W[e].T)
    del y
    g = swl.grouped_matmul_backward(dy, x, off, W)
    for rows, e in ((slice(5, 105), 1), (slice(cut - 50, cut), 1), (slice(cut, R), 2)):
        _product(g["dx"][rows], dy[rows], W[e])
    assert (g["dW"][0] == 0).all() and (g["db"][0] == 0).all()
    _product(g["dW"][2], dy[cut:].T, x[cut:])
    _close(g["db"][2], dy[cut:].double().sum(0), dy[cut:].double().abs().sum(0), R - cut)


@pytest.mark.parametrize("dtype", [F, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows", [6, 90])
def test_weights_past_32_bits(rows, dtype):
    K, O = 1024, 2048
    N = (1 << 31) // (K * O) + 3
    W = torch.empty((N, O, K), dtype=dtype, device="cuda")
    used = (0, N // 2, N - 1)
    for i, e in enumerate(used):
        W[e] = _n(10 + i, (O, K), dtype, K ** -0.5)
    x, dy = _n(4, (rows, K), dtype), _n(5, (rows, O), dtype, 0.1)
    third = rows // 3
    sizes = torch.zeros(N, dtype=torch.int64, device="cuda")
    for e in used:
        sizes[e] = third
    off = torch.cat([sizes.new_zeros(1), sizes.cumsum(0)]).to(torch.int32)
    y = swl.grouped_matmul(x, off, W)
    dx, dW = torch.zeros_like(x), torch.full_like(W, 7)
    swl.grouped_matmul_backward(dy, x, off, W, dx=dx, dW=dW)
    for i, e in enumerate(used):
        r = slice(i * third, (i + 1) * third)
        _product(y[r], x[r], W[e].T)
        _product(dx[r], dy[r], W[e])
        _product(dW[e], dy[r].T, x[r])
    assert (dW[1] == 0).all() and (dW[N - 2] == 0).all()


@pytest.mark.parametrize("dtype", [F, BF], ids=["f32", "bf16"])
def test_very_many_groups(dtype):
    N, K, O = 100003, 8, 8
    g = torch.Generator(device="cuda").manual_seed(6)
    sizes = torch.randint(0, 4, (N,), generator=g, device="cuda")
    off = torch.cat([sizes.new_zeros(1), sizes.cumsum(0)]).to(torch.int32)
    R = int(off[-1])
    e = torch.repeat_interleave(torch.arange(N, device="cuda"), sizes)
    x, dy, W = _n(7, (R, K), dtype), _n(8, (R, O), dtype), _n(9, (N, O, K), dtype)
    X, G, D = x.double(), dy.double(), W.double()[e]
    y, b = swl.grouped_matmul(x, off, W), swl.grouped_matmul_backward(dy, x, off, W)

    def bmm(p, q):
        return torch.einsum(p, *q), torch.einsum(p, *[t.abs() for t in q])

    _close(y, *bmm("rok,rk->ro", (D, X)), K)
    _close(b["dx"], *bmm("rok,ro->rk", (D, G)), O)
    outer, size = bmm("ro,rk->rok", (G, X))
    zero = torch.zeros((N, O, K), dtype=torch.float64, device="cuda")
    _close(b["dW"], zero.index_add(0, e, outer), zero.index_add(0, e, size), 4)
    zero = zero[:, :, 0]
    _close(b["db"], zero.index_add(0, e, G), zero.index_add(0, e, G.abs()), 4)


def _shifted(t):
    """The same values one element behind a 16-byte boundary."""
    flat = torch.full((t.numel() + 2,), float("nan"), dtype=t.dtype, device=t.device)
    flat[1:-1] = t.reshape(-1)
    return flat[1:-1].view(t.shape)


@pytest.mark.parametrize("K,O", [(64, 136), (66, 40), (65, 33)])
@pytest.mark.parametrize("rows", [7, 90])
def test_fp32_products_at_odd_addresses(rows, K, O):
    x, dy, W, b = (_n(i, s, F) for i, s in enumerate(((rows, K), (rows, O), (2, O, K), (2, O))))
    off = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device="cuda")
    for shift in range(16):
        t = [_shifted(q) if shift >> i & 1 else q for i, q in enumerate((x, dy, W, b))]
        out = _shifted(torch.zeros_like(dy))
        y = swl.grouped_matmul(t[0], off, t[2], bias=t[3], out=out)
        o = dict(dx=_shifted(torch.zeros_like(x)), dW=_shifted(torch.zeros_like(W)),
                 db=_shifted(torch.zeros_like(b)))
        g = swl.grouped_matmul_backward(t[1], t[0], off, t[2], **o)
        for e, r in enumerate((slice(0, rows // 3), slice(rows // 3, rows))):
            want = x[r].double() @ W[e].double().T + b[e].double()
            _close(y[r], want, x[r].double().abs() @ W[e].double().abs().T + b[e].double().abs(), K)
            _product(g["dx"][r], dy[r], W[e])
            _product(g["dW"][e], dy[r].T, x[r])
            _close(g["db"][e], dy[r].double().sum(0), dy[r].double().abs().sum(0), rows)


@pytest.mark.parametrize("dtype", [F, BF], ids=["f32", "bf16"])
def test_norms_past_32_bits_repeat_a_small_batch(dtype):
    """Rows far into a batch of 2^31 elements and more: equal to the same rows in a batch of
    their own, and column sums equal to those of the batch's only rows with gradients."""
    d = 2048
    T = (1 << 31) // d + 70
    x, y = _n(20, (70, d), dtype), _n(21, (70, d), dtype)
    gate = torch.rand(70, device="cuda")
    w, s = _n(22, (d,), F), _n(23, (d,), F)
    big_x, big_y = torch.zeros((T, d), dtype=dtype, device="cuda"), torch.zeros((T, d), dtype=dtype, device="cuda")
    big_gate = torch.zeros(T, device="cuda")
    big_x[-70:], big_y[-70:], big_gate[-70:] = x, y, gate
    args = dict(w_pre=w, w_post=w, scale=s)
    want = swl.norm_residual(x, y=y, gate=gate, **args)
    got = swl.norm_residual(big_x, y=big_y, gate=big_gate, **args)
    tol = 2.0 ** -7 if dtype == BF else 2.0 ** -20      # (the batch's size chooses the sums' order)
    for k in ("r", "h"):
        assert ((got[k][-70:].float() - want[k].float()).abs() <= tol * (1 + want[k].float().abs())).all(), k
        assert (got[k][:64] == 0).all(), k
    r = got["r"]
    del got
    dr, dh = _n(24, (70, d), dtype), _n(25, (70, d), dtype)
    want = swl.norm_residual_backward(dr, dh, r[-70:].contiguous(), y=y, gate=gate, **args)
    big_dr, big_dh = torch.zeros_like(big_x), torch.zeros_like(big_x)
    big_dr[-70:], big_dh[-70:] = dr, dh
    got = swl.norm_residual_backward(big_dr, big_dh, r, y=big_y, gate=big_gate, **args)
    for k in ("dx", "dy", "dgate"):
        a, b = got[k][-70:].float(), want[k].float()
        assert ((a - b).abs() <= tol * (b.abs() + b.abs().mean())).all(), k
        assert (got[k][:64] == 0).all(), k
    for k in ("dw_pre", "dw_post", "dscale"):
        a, b = got[k].double(), want[k].double()
        assert ((a - b).abs() <= 2.0 ** -16 * (b.abs() + b.abs().mean())).all(), k
