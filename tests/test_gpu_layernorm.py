"""The layer norm, its quantized outputs and its gradients.

Values against the definition in 64 bits; codes, scales and amax bit for bit
against the oracle on the kernel's own FP32 y; gradients against the formula
and against differences. Tolerances: a sum whose terms pass at most d additions
each has relative error d U of the sum of magnitudes; d is the lane's share of
the row and the tree over lanes and waves.
"""
import math

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
    n = math.prod(shape)
    buf = torch.empty(n + 8, dtype=dtype, device=DEV)[shift:shift + n]
    buf.copy_(torch.randn(n, generator=g).to(dtype))
    return buf.view(*shape)


def half(dtype):
    return U if dtype == FP else 2.0 ** -8


def plain(x, res, w, b):
    """h, mean, rstd, y and the bounds of the last three's FP32 errors, in 64 bits.

    The first mean mu0 is off by e0 = (d + 1) U mean|h|. From it, d_k = h_k - mu0 (one rounding of d_k) is summed to
    dm, off by (d + 2) U mean|d_k|, which mean = mu0 + dm rounds once more. d_k - dm is off by that and two roundings;
    the variance, a sum of squares, by (d + 4) U relative, and by dm's share, of the same order; rstd by half of it."""
    K = x.shape[1]
    h = np64(x) + (0 if res is None else np64(res))
    mu = h.mean(1)
    d = h - mu[:, None]
    var = (d * d).mean(1)
    r = 1 / np.sqrt(var + EPS)
    size = np.abs(d).mean(1)
    e0 = (depth(K) + 2) * U * np.abs(h).mean(1) + U * np.abs(h).max(1)  # (h itself is rounded to FP32)
    em = (depth(K) + 4) * U * (size + e0) + U * np.abs(mu) + U * np.abs(h).max(1)
    # variance: relative (d + 6) U, and h's own rounding, 2 |d| U |h|
    rv = ((depth(K) + 6) * U * var + 2 * U * (np.abs(d) * np.abs(h)).mean(1) + (depth(K) + 6) * U * e0 ** 2) / (var + EPS)
    er = (0.5 * rv + 3 * U) * r
    w64, b64 = np64(w), np.zeros(K) if b is None else np64(b)
    y = d * r[:, None] * w64 + b64
    ed = em[:, None] + U * np.abs(h) + 2 * U * (np.abs(d) + e0[:, None])
    ey = (ed * r[:, None] + np.abs(d) * er[:, None] + U * np.abs(d) * r[:, None]) * 1.001 * np.abs(w64) + U * np.abs(y)
    return h, mu, r, y, em, er, ey


CASES = [(1, 1), (2, 7), (3, 8), (5, 15), (4, 16), (3, 31), (40, 120), (17, 128), (5, 130), (1, 8192), (7, 512), (5, 513), (3, 2048),
         (2, 2881), (3, 4096), (2, 4104), (2, 8193), (2, 16384), (2, 16400), (1, 28672), (1, 32768), (2, 32769), (1, 50001)]


def rows(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, FP), (FP, FP), (FP, BF)])
@pytest.mark.parametrize("M,K", CASES)
def test_forward(M, K, dtype, wdtype):
    say(f"[gpu] layer norm {M}x{K} {dtype} {wdtype}")
    g = torch.Generator().manual_seed(M * 31 + K)
    x = (rand(g, M, K) + 3 * rand(g, M, 1)).to(dtype)
    res, w, b = rand(g, M, K, dtype=dtype), rand(g, K, dtype=wdtype), rand(g, K, dtype=wdtype)
    for r_, b_ in ((None, None), (res, b)):
        h64, mu64, r64, y64, em, er, ey = plain(x, r_, w, b_)
        h, y = torch.empty_like(x), torch.empty(M, K, device=DEV)
        mean, rstd, amax = (torch.empty(M, device=DEV) for _ in range(3))
        q8 = torch.empty(M, K, dtype=torch.float8_e4m3fn, device=DEV)
        p.nvfp4_layernorm(x, w, EPS, bias=b_, residual=r_, h=h, y=y, mean=mean, rstd=rstd, q=q8, row_amax=amax)
        torch.cuda.synchronize()
        # the stored sum: FP32 addition, then one rounding to the type
        assert torch.equal(h, (x.float() + (0 if r_ is None else r_.float())).to(dtype))
        assert np.all(np.abs(np64(mean) - mu64) <= em)
        assert np.all(np.abs(np64(rstd) - r64) <= er)
        assert np.all(np.abs(np64(y) - y64) <= ey)
        assert torch.equal(amax, y.abs().amax(1))
        # codes of that y: RN(y RN(top / a)), to nearest even
        yc, ac = y.cpu(), amax.cpu()
        enc = lambda top: torch.where(ac > 0, torch.full_like(ac, top) / ac, torch.ones_like(ac))[:, None]
        want8 = (yc * enc(448.0)).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(q8.view(torch.uint8).cpu(), want8.view(torch.uint8))
        qi, ai = torch.empty(M, K, dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
        p.nvfp4_layernorm(x, w, EPS, bias=b_, residual=r_, q=qi, row_amax=ai)
        assert torch.equal(ai, amax)
        assert torch.equal(qi.cpu(), torch.round(yc * enc(127.0)).clamp(-127, 127).to(torch.int8))
        qs, as_ = torch.empty_like(qi), torch.empty_like(ai)
        p.nvfp4_int8_quantize(y, as_, qs)   # and the quantizer's codes of it
        assert torch.equal(qs, qi) and torch.equal(as_, ai)
        for bound in (448.0, 256.0):
            q4 = torch.full((M, (K + 1) // 2), 0xEE, dtype=torch.uint8, device=DEV)
            s4 = torch.full((M, (K + 15) // 16), 0xEE, dtype=torch.uint8, device=DEV)
            yb, a4 = torch.empty(M, K, dtype=BF, device=DEV), torch.empty(M, device=DEV)
            p.nvfp4_layernorm(x, w, EPS, bias=b_, residual=r_, y=yb, q=q4, s=s4, row_amax=a4, bound=bound)
            torch.cuda.synchronize()
            assert torch.equal(a4, amax) and torch.equal(yb, y.to(BF))
            oq, os_ = oracle.quantize_rowwise(y.cpu().numpy(), oracle.MODE_LINE, amax.cpu().numpy(), bound)
            assert torch.equal(q4, rows(oq)) and torch.equal(s4, rows(os_))


@pytest.mark.parametrize("K", [100, 512, 2881, 8192, 28672, 40000])
def test_a_mean_far_from_zero(K):
    """Rows 1 wide around means up to 3e4: what FP32 holds of the rows themselves is all that is lost."""
    say(f"[gpu] layer norm far means {K}")
    g = torch.Generator().manual_seed(K)
    x = rand(g, 4, K) + torch.tensor([[0.0], [100.0], [-3e4], [1e3]], device=DEV)
    x[3] = 1e3                                    # a constant row: variance 0
    w = torch.ones(K, device=DEV)
    h64, mu64, r64, y64, em, er, ey = plain(x, None, w, None)
    y, mean, rstd = torch.empty(4, K, device=DEV), torch.empty(4, device=DEV), torch.empty(4, device=DEV)
    p.nvfp4_layernorm(x, w, EPS, y=y, mean=mean, rstd=rstd)
    assert np.all(np.abs(np64(mean) - mu64) <= em) and np.all(np.abs(np64(rstd) - r64) <= er)
    assert np.all(np.abs(np64(y) - y64) <= ey)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("K", [24, 300, 2880, 9000, 40000])
def test_any_address_and_in_place(K, dtype):
    g = torch.Generator().manual_seed(K)
    for shift in (1, 2, 3):
        x, res, w, b = (rand(g, *s, dtype=dtype, shift=shift) for s in ((3, K), (3, K), (K,), (K,)))
        x0, res0, w0, b0 = x.clone(), res.clone(), w.clone(), b.clone()
        h, y = torch.empty_like(x0), torch.empty(3, K, device=DEV)
        p.nvfp4_layernorm(x0, w0, EPS, bias=b0, residual=res0, h=h, y=y)
        y2 = torch.full((3 * K + 4,), 5.0, device=DEV)
        view = y2[shift:shift + 3 * K].view(3, K)
        p.nvfp4_layernorm(x, w, EPS, bias=b, residual=res, h=res, y=view)
        assert torch.equal(res, h) and torch.equal(view, y)
        assert bool((y2[:shift] == 5.0).all()) and bool((y2[shift + 3 * K:] == 5.0).all())
        res = res0.clone()
        p.nvfp4_layernorm(x, w, EPS, bias=b, residual=res, h=x, y=view)
        assert torch.equal(x, h) and torch.equal(view, y)


@pytest.mark.parametrize("K", [96, 300, 2881, 8192, 28672, 40000])
def test_infinities_and_nan(K):
    """A row that holds one is NaN throughout, statistics and amax too; other rows keep their bits."""
    M = 6
    x, w, b = torch.randn(M, K, device=DEV), torch.randn(K, device=DEV), torch.randn(K, device=DEV)

    def run(x):
        o = dict(h=torch.empty_like(x), y=torch.empty_like(x), mean=torch.empty(M, device=DEV), rstd=torch.empty(M, device=DEV),
                 q=torch.empty(M, K, dtype=torch.int8, device=DEV), row_amax=torch.empty(M, device=DEV))
        p.nvfp4_layernorm(x, w, EPS, bias=b, **o)
        return o
    o0 = run(x)
    x2 = x.clone()
    x2[1, 7], x2[2, K - 1], x2[4, K // 2] = float("nan"), float("inf"), -float("inf")
    o = run(x2)
    for k in o:
        assert torch.equal(o[k][[0, 3, 5]], o0[k][[0, 3, 5]]), k
    for k in ("y", "mean", "rstd", "row_amax"):
        assert bool(torch.isnan(o[k][[1, 2, 4]]).all()), k


def backward64(dy, h, mu, r, w, dres):
    xh = (h - mu[:, None]) * r[:, None]
    g = dy * w
    m1, m2 = g.mean(1, keepdims=True), (g * xh).mean(1, keepdims=True)
    dx = r[:, None] * (g - m1 - xh * m2)
    return dx + (0 if dres is None else dres), (dy * xh).sum(0), dy.sum(0), xh, g, m1, m2


BWD = [(1, 1), (3, 7), (40, 16), (2100, 96), (1500, 128), (5, 130), (700, 512), (2, 513), (1100, 2048), (5, 2881), (700, 4096), (9, 8193),
       (600, 8192), (3, 16384), (300, 16384), (3, 28672), (300, 17000), (2, 40001)]


@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (FP, FP), (BF, FP), (FP, BF)])
@pytest.mark.parametrize("M,K", BWD)
def test_backward(M, K, dtype, wdtype):
    say(f"[gpu] layer norm bwd {M}x{K} {dtype} {wdtype}")
    g = torch.Generator().manual_seed(M + K)
    dy, dres, w = rand(g, M, K, dtype=dtype), rand(g, M, K, dtype=dtype), rand(g, K, dtype=wdtype)
    h = (rand(g, M, K) + 3 * rand(g, M, 1)).to(dtype)
    mu = h.float().mean(1)
    r = torch.rsqrt((h.float() - mu[:, None]).square().mean(1) + EPS)
    for d_ in (None, dres):
        dx64, dw64, db64, xh, gg, m1, m2 = backward64(np64(dy), np64(h), np64(mu), np64(r), np64(w), None if d_ is None else np64(d_))
        dx = torch.full_like(dy, float("nan"))
        dw, db = torch.full((K,), float("nan"), device=DEV), torch.full((K,), float("nan"), device=DEV)
        p.nvfp4_layernorm_backward(dy, h, w, mu, r, dx, dweight=dw, dbias=db, dres=d_)
        torch.cuda.synchronize()
        # the means' terms pass depth(K) additions; xh, g and what joins them a handful of roundings
        n = depth(K) + 6
        err = np64(r)[:, None] * (n * U * (np.abs(gg).mean(1, keepdims=True) + np.abs(xh) * np.abs(gg * xh).mean(1, keepdims=True))
                                  + 4 * U * (np.abs(gg) + np.abs(m1) + np.abs(xh * m2)))
        err = err + 2 * U * np.abs(dx64)
        assert np.all(np.abs(np64(dx) - dx64) <= err + half(dtype) * (np.abs(dx64) + err))
        assert np.all(np.abs(np64(dw) - dw64) <= (M + 6) * U * np.abs(np64(dy) * xh).sum(0) + 1e-45)
        assert np.all(np.abs(np64(db) - db64) <= (M + 4) * U * np.abs(np64(dy)).sum(0) + 1e-45)
        # without the sums, or with one of them: the same bits
        for kw in (dict(), dict(dweight=torch.empty(K, device=DEV)), dict(dbias=torch.empty(K, device=DEV))):
            dx2 = torch.empty_like(dx)
            p.nvfp4_layernorm_backward(dy, h, w, mu, r, dx2, dres=d_, **kw)
            assert torch.equal(dx, dx2)
            for k, v in kw.items():
                assert torch.equal(v, dw if k == "dweight" else db)
        at = dy.clone() if d_ is None else d_.clone()           # dx over dy, or over dres
        dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
        p.nvfp4_layernorm_backward(at if d_ is None else dy, h, w, mu, r, at, dweight=dw2, dbias=db2, dres=None if d_ is None else at)
        assert torch.equal(at, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M,K", [(1, 24), (40, 100), (5, 513), (5, 2880), (5, 9000), (3, 28000), (3, 40000)])
def test_backward_at_any_address(M, K, dtype):
    g = torch.Generator().manual_seed(K)
    for shift in (1, 2, 3):
        def at(*s, dt=dtype):
            n = math.prod(s)
            buf = torch.full((n + 8,), 5.0, device=DEV, dtype=dt)
            buf[shift:shift + n] = torch.randn(n, generator=g).to(DEV).to(dt)
            return buf, buf[shift:shift + n].view(*s)
        (_, dy), (_, h), (_, dres), (_, w), (_, mu), (_, r) = at(M, K), at(M, K), at(M, K), at(K), at(M, dt=FP), at(M, dt=FP)
        (bx, dx), (bw, dw), (bb, db) = at(M, K), at(K, dt=FP), at(K, dt=FP)
        want, wantw, wantb = torch.empty(M, K, device=DEV, dtype=dtype), torch.empty(K, device=DEV), torch.empty(K, device=DEV)
        p.nvfp4_layernorm_backward(*(t.clone() for t in (dy, h, w, mu, r)), want, dweight=wantw, dbias=wantb, dres=dres.clone())
        p.nvfp4_layernorm_backward(dy, h, w, mu, r, dx, dweight=dw, dbias=db, dres=dres)
        assert torch.equal(dx, want) and torch.equal(dw, wantw) and torch.equal(db, wantb)
        for buf in (bx, bw, bb):
            n = buf.numel() - 8
            assert bool((buf[:shift] == 5.0).all()) and bool((buf[shift + n:] == 5.0).all())


def test_backward_against_differences():
    """Central differences of the 64-bit forward pass: dL for L = sum(y t)."""
    rng = np.random.RandomState(0)
    M, K = 3, 40
    x, w, b, t = (a.astype(np.float32).astype(np.float64) for a in
                  (rng.standard_normal((M, K)) + 1, rng.standard_normal(K), rng.standard_normal(K), rng.standard_normal((M, K))))

    def loss(x, w, b):
        d = x - x.mean(1, keepdims=True)
        return ((d / np.sqrt((d * d).mean(1, keepdims=True) + EPS) * w + b) * t).sum()
    e = 1e-5
    dxn, dwn, dbn = np.empty((M, K)), np.empty(K), np.empty(K)
    for i in range(M):
        for k in range(K):
            d = np.zeros((M, K))
            d[i, k] = e
            dxn[i, k] = (loss(x + d, w, b) - loss(x - d, w, b)) / (2 * e)
    for k in range(K):
        d = np.zeros(K)
        d[k] = e
        dwn[k] = (loss(x, w + d, b) - loss(x, w - d, b)) / (2 * e)
        dbn[k] = (loss(x, w, b + d) - loss(x, w, b - d)) / (2 * e)
    f = lambda a: torch.from_numpy(a.astype(np.float32)).to(DEV)
    mean, rstd = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    p.nvfp4_layernorm(f(x), f(w), EPS, bias=f(b), mean=mean, rstd=rstd)
    dx, dw, db = torch.empty(M, K, device=DEV), torch.empty(K, device=DEV), torch.empty(K, device=DEV)
    p.nvfp4_layernorm_backward(f(t), f(x), f(w), mean, rstd, dx, dweight=dw, dbias=db)
    # differences: e^2 of the third derivative and 1e-16 / e of rounding, far below 1e-6
    for got, want in ((dx, dxn), (dw, dwn), (db, dbn)):
        assert np.abs(np64(got) - want).max() < 1e-5


@pytest.mark.parametrize("K", [96, 300, 2881, 8192, 28672, 40000])
def test_gradient_of_rows_with_nan(K):
    M = 5
    dy, h, w = torch.randn(M, K, device=DEV), torch.randn(M, K, device=DEV), torch.randn(K, device=DEV)
    mu, r = torch.randn(M, device=DEV), torch.rand(M, device=DEV) + 0.5

    def run(dy):
        dx, dw, db = torch.empty_like(dy), torch.empty(K, device=DEV), torch.empty(K, device=DEV)
        p.nvfp4_layernorm_backward(dy, h, w, mu, r, dx, dweight=dw, dbias=db)
        return dx, dw, db
    dx0, dw0, db0 = run(dy)
    dy2 = dy.clone()
    dy2[2, 5] = float("nan")
    dx, dw, db = run(dy2)
    ok = torch.arange(K, device=DEV) != 5
    assert torch.equal(dx[[0, 1, 3, 4]], dx0[[0, 1, 3, 4]]) and bool(torch.isnan(dx[2]).all())
    for a, a0 in ((dw, dw0), (db, db0)):
        assert torch.equal(a[ok], a0[ok]) and bool(torch.isnan(a[5]))


def test_more_rows_than_a_launch_holds():
    """2^20 rows a launch: the ones after it, and the ones before, as calls of their own give them."""
    M, K = (1 << 20) + 5, 40
    g = torch.Generator(device=DEV).manual_seed(1)
    x, w = torch.randn(M, K, generator=g, device=DEV), torch.randn(K, generator=g, device=DEV)

    def run(x):
        n = x.shape[0]
        o = dict(y=torch.empty_like(x), mean=torch.empty(n, device=DEV), rstd=torch.empty(n, device=DEV), row_amax=torch.empty(n, device=DEV),
                 q=torch.empty(n, K, dtype=torch.int8, device=DEV))
        p.nvfp4_layernorm(x, w, EPS, bias=w, **o)
        q, a = torch.empty_like(o["q"]), torch.empty(n, device=DEV)
        p.nvfp4_int8_quantize(x, a, q)
        return dict(o, q2=q, a2=a)
    whole = run(x)
    for lo, hi in ((0, 1000), ((1 << 20) - 3, M)):
        for k, v in run(x[lo:hi].clone()).items():
            assert torch.equal(whole[k][lo:hi], v), (k, lo)


def test_noop_stream_and_replay():
    g = torch.Generator().manual_seed(5)
    for M, K in ((64, 4096), (500, 96)):
        x, res, w, b = rand(g, M, K, dtype=BF), rand(g, M, K, dtype=BF), rand(g, K, dtype=BF), rand(g, K, dtype=BF)
        q = torch.empty(M, K, dtype=torch.int8, device=DEV)
        h, dx = torch.empty_like(x), torch.empty_like(x)
        mean, rstd, amax = (torch.empty(M, device=DEV) for _ in range(3))
        dw, db = torch.empty(K, device=DEV), torch.empty(K, device=DEV)
        ws = torch.empty(p.nvfp4_layernorm_backward_workspace(M, K), dtype=torch.uint8, device=DEV)
        outs = (q, h, mean, rstd, amax, dx, dw, db)

        def call(noop=None, stream=None):
            p.nvfp4_layernorm(x, w, EPS, bias=b, residual=res, h=h, mean=mean, rstd=rstd, q=q, row_amax=amax, noop=noop, stream=stream)
            p.nvfp4_layernorm_backward(x, h, w, mean, rstd, dx, dweight=dw, dbias=db, dres=res, workspace=ws, noop=noop, stream=stream)
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
    q8 = torch.empty(4, 32, dtype=torch.int8, device=DEV)
    q4 = torch.empty(4, 16, dtype=torch.uint8, device=DEV)
    s4 = torch.empty(4, 2, dtype=torch.uint8, device=DEV)
    for kw in (dict(), dict(q=q8), dict(q=q4, row_amax=f), dict(q=q4, s=s4, row_amax=f, bound=0.0), dict(q=q8, s=s4, row_amax=f)):
        with pytest.raises(p.Nvfp4Error):
            p.nvfp4_layernorm(x, w, EPS, **kw)
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(p.Nvfp4Error):
            p.nvfp4_layernorm(x, w, eps, y=y)
    for kw in (dict(y=y.cpu()), dict(h=y[:3]), dict(rstd=f[:3]), dict(mean=f[:3]), dict(residual=y.t().contiguous().t()),
               dict(y=y, bias=w[:31])):
        with pytest.raises(ValueError):
            p.nvfp4_layernorm(x, w, EPS, **kw)
    for kw in (dict(y=y, bias=w.bfloat16()), dict(q=q8.short(), row_amax=f), dict(y=y.half())):
        with pytest.raises((TypeError, KeyError)):
            p.nvfp4_layernorm(x, w, EPS, **kw)
    with pytest.raises(TypeError):
        p.nvfp4_layernorm(x.half(), w, EPS, y=y)
    for kw in (dict(dweight=w[:31]), dict(dbias=w[:31]), dict(dweight=w.clone(), workspace=f), dict(dbias=w.clone(), workspace=f)):
        with pytest.raises(ValueError):
            p.nvfp4_layernorm_backward(x, x, w, f, f, y, **kw)
    with pytest.raises(TypeError):
        p.nvfp4_layernorm_backward(x, x.bfloat16(), w, f, f, y)
