"""The root-mean-square norm, its quantized outputs and its gradient.

y against the definition in 64 bits; codes, scales and amax bit for bit
against the oracle on the kernel's own FP32 y; gradients against the formula
and against differences. Tolerances: a sum of squares whose terms pass at most
d additions each has relative error d 2^-24, halved by the square root; d is
the lane's share of the row and the tree over lanes and waves.
"""
import numpy as np
import pytest
import torch

import oracle
import precision_quantization_row_amd as p
from parity_utils import say
from product_utils import DEV, np64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5
BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    p.load_library()


def depth(K):
    return 8 * (K // 512 + 1) + 24


def rand(g, *shape, dtype=FP, shift=0):
    n = int(np.prod(shape))
    buf = torch.empty(n + 8, dtype=dtype, device=DEV)[shift:shift + n]
    buf.copy_(torch.randn(n, generator=g).to(dtype))
    return buf.view(*shape)


def half(dtype):
    return 2.0 ** -24 if dtype == FP else 2.0 ** -8


def plain(x, res, w):
    h = np64(x) + (0 if res is None else np64(res))
    r = 1 / np.sqrt((h * h).mean(1) + EPS)
    return h, r, h * r[:, None] * np64(w)


def rows(oracle_bytes):
    return torch.from_numpy(np.ascontiguousarray(oracle_bytes)).to(DEV)


CASES = [(1, 1), (2, 7), (3, 8), (5, 15), (4, 16), (3, 31), (1, 8192), (7, 512), (5, 513), (3, 2048), (2, 2881),
         (3, 4096), (2, 4104), (2, 8193), (2, 16384), (2, 16400), (1, 28672), (1, 32768), (2, 32769), (1, 50001)]


@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, FP), (FP, FP), (FP, BF)])
@pytest.mark.parametrize("M,K", CASES)
def test_forward(M, K, dtype, wdtype):
    say(f"[gpu] norm {M}x{K} {dtype} {wdtype}")
    g = torch.Generator().manual_seed(M * 31 + K)
    x, res, w = rand(g, M, K, dtype=dtype), rand(g, M, K, dtype=dtype), rand(g, K, dtype=wdtype)
    for r_ in (None, res):
        h64, r64, y64 = plain(x, r_, w)
        h = torch.empty_like(x)
        y = torch.empty(M, K, device=DEV)
        rstd, amax = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
        q8 = torch.empty(M, K, dtype=torch.float8_e4m3fn, device=DEV)
        p.nvfp4_rmsnorm(x, w, EPS, residual=r_, h=h, y=y, rstd=rstd, q=q8, row_amax=amax)
        torch.cuda.synchronize()
        # the stored sum: FP32 addition, then one rounding to the type
        want_h = (x.float() + (0 if r_ is None else r_.float())).to(dtype)
        assert torch.equal(h, want_h)
        rel = (depth(K) / 2 + 8) * U
        assert np.all(np.abs(np64(rstd) - r64) <= rel * r64)
        # h itself carries one rounding, the products two more
        assert np.all(np.abs(np64(y) - y64) <= (rel + 4 * U) * np.abs(y64) + U * np.abs(h64 * r64[:, None] * np64(w)))
        assert torch.equal(amax, y.abs().amax(1))
        # 8-bit codes of that y: RN(y * RN(448 / a)), round to nearest even
        yc, ac = y.cpu(), amax.cpu()
        enc = torch.where(ac > 0, torch.full_like(ac, 448.0) / ac, torch.ones_like(ac))
        want8 = (yc * enc[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(q8.view(torch.uint8).cpu(), want8.view(torch.uint8))
        # 4-bit codes of that y: the oracle's rowwise copy; BF16 y: the FP32 y rounded
        for bound in (448.0, 256.0):
            q4 = torch.full((M, (K + 1) // 2), 0xEE, dtype=torch.uint8, device=DEV)
            s4 = torch.full((M, (K + 15) // 16), 0xEE, dtype=torch.uint8, device=DEV)
            yb, amax4 = torch.empty(M, K, dtype=BF, device=DEV), torch.empty(M, device=DEV)
            p.nvfp4_rmsnorm(x, w, EPS, residual=r_, y=yb, q=q4, s=s4, row_amax=amax4, bound=bound)
            torch.cuda.synchronize()
            assert torch.equal(amax4, amax) and torch.equal(yb, y.to(BF))
            oq, os_ = oracle.quantize_rowwise(y.cpu().numpy(), oracle.MODE_LINE, amax.cpu().numpy(), bound)
            assert torch.equal(q4, rows(oq)) and torch.equal(s4, rows(os_))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("K", [24, 2880, 9000])
def test_any_address_and_in_place(K, dtype):
    g = torch.Generator().manual_seed(K)
    for shift in (1, 2, 3):
        x, res, w = (rand(g, *s, dtype=dtype, shift=shift) for s in ((3, K), (3, K), (K,)))
        x0, res0, w0 = x.clone(), res.clone(), w.clone()
        h, y = torch.empty_like(x0), torch.empty(3, K, device=DEV)
        p.nvfp4_rmsnorm(x0, w0, EPS, residual=res0, h=h, y=y)
        y2 = torch.full((3 * K + 4,), 5.0, device=DEV)
        p.nvfp4_rmsnorm(x, w, EPS, residual=res, h=res, y=y2[shift:shift + 3 * K].view(3, K))
        assert torch.equal(res, h) and torch.equal(y2[shift:shift + 3 * K].view(3, K), y)
        assert torch.all(y2[:shift] == 5.0) and torch.all(y2[shift + 3 * K:] == 5.0)


def test_rows_of_zeros_and_extremes():
    for K in (16, 4097, 40000):
        x = torch.zeros(4, K, device=DEV)
        x[1, 0] = 1e18            # its square is near the top of FP32
        x[2] = 1e-30              # squares underflow: eps alone
        x[3, K - 1] = -3.0
        w = torch.ones(K, device=DEV)
        y, rstd, amax = torch.empty(4, K, device=DEV), torch.empty(4, device=DEV), torch.empty(4, device=DEV)
        q = torch.empty(4, (K + 1) // 2, dtype=torch.uint8, device=DEV)
        s = torch.empty(4, (K + 15) // 16, dtype=torch.uint8, device=DEV)
        p.nvfp4_rmsnorm(x, w, EPS, y=y, rstd=rstd, q=q, s=s, row_amax=amax)
        h64, r64, y64 = plain(x, None, w)
        assert np.all(np.abs(np64(y) - y64) <= (depth(K) / 2 + 12) * U * np.abs(y64) + 1e-45)
        assert torch.all(y[0] == 0) and torch.all(q[0] == 0) and float(amax[0]) == 0.0
        oq, os_ = oracle.quantize_rowwise(y.cpu().numpy(), oracle.MODE_LINE, amax.cpu().numpy(), 448.0)
        assert torch.equal(q, rows(oq)) and torch.equal(s, rows(os_))


def backward64(dy, h, r, w, dres):
    xh = h * r[:, None]
    g = dy * w
    dx = r[:, None] * (g - xh * (g * xh).mean(1, keepdims=True))
    return dx + (0 if dres is None else dres), (dy * xh).sum(0)


BWD = [(1, 1), (3, 7), (40, 16), (2, 513), (1500, 96), (5, 2881), (700, 4096), (9, 8193), (3, 16384), (3, 28672),
       (2, 40001)]


@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (FP, FP), (BF, FP)])
@pytest.mark.parametrize("M,K", BWD)
def test_backward(M, K, dtype, wdtype):
    say(f"[gpu] norm bwd {M}x{K} {dtype} {wdtype}")
    g = torch.Generator().manual_seed(M + K)
    dy, h, dres = (rand(g, M, K, dtype=dtype) for _ in range(3))
    w = rand(g, K, dtype=wdtype)
    r = torch.rsqrt(h.float().square().mean(1) + EPS)
    for d_ in (None, dres):
        dx64, dw64 = backward64(np64(dy), np64(h), np64(r), np64(w), None if d_ is None else np64(d_))
        dx, dw = torch.full_like(dy, float("nan")), torch.full((K,), float("nan"), device=DEV)
        p.nvfp4_rmsnorm_backward(dy, h, w, r, dx, dweight=dw, dres=d_)
        torch.cuda.synchronize()
        xh, gg = np64(h) * np64(r)[:, None], np64(dy) * np64(w)
        # the mean's terms pass depth(K) additions; then a handful of roundings
        err = np64(r)[:, None] * ((depth(K) + 6) * U * np.abs(xh) * np.abs(gg * xh).mean(1, keepdims=True)
                                  + 4 * U * np.abs(gg))
        err = err + 2 * U * np.abs(dx64)
        assert np.all(np.abs(np64(dx) - dx64) <= err + half(dtype) * (np.abs(dx64) + err))
        assert np.all(np.abs(np64(dw) - dw64) <= (M + 4) * U * np.abs(np64(dy) * xh).sum(0) + 1e-45)
        dx2 = torch.empty_like(dx)
        p.nvfp4_rmsnorm_backward(dy, h, w, r, dx2, dres=d_)   # without dweight; the same bits
        assert torch.equal(dx, dx2)
        inplace = dy.clone() if d_ is None else d_.clone()
        dw2 = torch.empty_like(dw)
        p.nvfp4_rmsnorm_backward(inplace if d_ is None else dy, h, w, r, inplace, dweight=dw2,
                                 dres=None if d_ is None else inplace)
        assert torch.equal(inplace, dx) and torch.equal(dw2, dw)


def test_backward_against_differences():
    """Central differences of the 64-bit forward pass: dL for L = sum(y * t)."""
    rng = np.random.RandomState(0)
    M, K = 3, 40
    x, w, t = rng.standard_normal((M, K)), rng.standard_normal(K), rng.standard_normal((M, K))
    x, w, t = (a.astype(np.float32).astype(np.float64) for a in (x, w, t))

    def loss(x, w):
        return (x / np.sqrt((x * x).mean(1, keepdims=True) + EPS) * w * t).sum()

    e = 1e-5
    dxn, dwn = np.empty((M, K)), np.empty(K)
    for i in range(M):
        for k in range(K):
            d = np.zeros((M, K))
            d[i, k] = e
            dxn[i, k] = (loss(x + d, w) - loss(x - d, w)) / (2 * e)
    for k in range(K):
        d = np.zeros(K)
        d[k] = e
        dwn[k] = (loss(x, w + d) - loss(x, w - d)) / (2 * e)
    f = lambda a: torch.from_numpy(a.astype(np.float32)).to(DEV)
    rstd, y = torch.empty(M, device=DEV), torch.empty(M, K, device=DEV)
    p.nvfp4_rmsnorm(f(x), f(w), EPS, y=y, rstd=rstd)
    dx, dw = torch.empty(M, K, device=DEV), torch.empty(K, device=DEV)
    p.nvfp4_rmsnorm_backward(f(t), f(x), f(w), rstd, dx, dweight=dw)
    # differences: e^2 of the third derivative and 1e-16 / e of rounding, far below 1e-6
    assert np.abs(np64(dx) - dxn).max() < 1e-5 and np.abs(np64(dw) - dwn).max() < 1e-5


def test_noop_stream_and_replay():
    g = torch.Generator().manual_seed(5)
    M, K = 64, 4096
    x, res, w = rand(g, M, K, dtype=BF), rand(g, M, K, dtype=BF), rand(g, K, dtype=BF)
    q = torch.empty(M, K, dtype=torch.float8_e4m3fn, device=DEV)
    h, rstd, amax = torch.empty_like(x), torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    dx, dw = torch.empty_like(x), torch.empty(K, device=DEV)
    ws = torch.empty(p.nvfp4_rmsnorm_backward_workspace(M, K), dtype=torch.uint8, device=DEV)
    outs = (q.view(torch.uint8), h, rstd, amax, dx, dw)

    def call(noop=None, stream=None):
        p.nvfp4_rmsnorm(x, w, EPS, residual=res, h=h, rstd=rstd, q=q, row_amax=amax, noop=noop, stream=stream)
        p.nvfp4_rmsnorm_backward(x, h, w, rstd, dx, dweight=dw, dres=res, workspace=ws, noop=noop, stream=stream)

    for t in outs:
        t.fill_(3)
    call(noop=torch.ones(1, device=DEV))
    assert all(bool((t == 3).all()) for t in outs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(4):
        x.copy_(torch.randn(M, K, generator=g).to(BF))
        call()
        want = [t.clone() for t in outs]
        for t in outs:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_refusals():
    x, w = torch.zeros(4, 32, device=DEV), torch.ones(32, device=DEV)
    y, f = torch.empty(4, 32, device=DEV), torch.empty(4, device=DEV)
    q8 = torch.empty(4, 32, dtype=torch.float8_e4m3fn, device=DEV)
    q4 = torch.empty(4, 16, dtype=torch.uint8, device=DEV)
    for kw in (dict(), dict(q=q8), dict(q=q4, row_amax=f), dict(q=q4, s=q4[:, :2].contiguous(), row_amax=f, bound=0.0),
               dict(q=q8, s=q4[:, :2].contiguous(), row_amax=f)):
        with pytest.raises(p.Nvfp4Error):
            p.nvfp4_rmsnorm(x, w, EPS, **kw)
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(p.Nvfp4Error):
            p.nvfp4_rmsnorm(x, w, eps, y=y)
    for kw in (dict(y=y.cpu()), dict(h=y[:3]), dict(rstd=f[:3]), dict(residual=y.t().contiguous().t())):
        with pytest.raises(ValueError):
            p.nvfp4_rmsnorm(x, w, EPS, **kw)
    with pytest.raises(ValueError):
        p.nvfp4_rmsnorm(x, w[:31], EPS, y=y)
    with pytest.raises(TypeError):
        p.nvfp4_rmsnorm(x.half(), w, EPS, y=y)
    with pytest.raises(ValueError):
        p.nvfp4_rmsnorm_backward(x, x, w, f, y, dweight=torch.empty(31, device=DEV))
    with pytest.raises(ValueError):
        p.nvfp4_rmsnorm_backward(x, x, w, f, y, dweight=w.clone(), workspace=f)
    with pytest.raises(TypeError):
        p.nvfp4_rmsnorm_backward(x, x.bfloat16(), w, f, y)
