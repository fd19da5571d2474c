"""The integer lines and product, the layer norm and the cache where a caller may bring them: through the short and
the long way of the binding, on other streams, in two graphs, with more elements than 32 bits count.

Everything bit for bit, against the same entry points' own smaller calls, or codes that the host computes alike.
"""
import numpy as np
import pytest
import torch

import precision_quantization_row_amd as p
from parity_utils import say
from product_utils import DEV
from test_gpu_int8 import codes

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
LINE = p.NVFP4_AMAX_LINE
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    p.load_library()


class Long:
    """Stands in for the native binding: every call takes the long way."""

    def __getattr__(self, name):
        return lambda *a: None


def everything(stream=None):
    """One call of each entry point; all outputs."""
    g = torch.Generator().manual_seed(1)
    t = lambda *s, dt=BF: torch.randn(*s, generator=g).to(dt).to(DEV)
    e = lambda *s, dt=FP: torch.full(s, 3, dtype=dt, device=DEV)
    M, K, N, H, D = 37, 264, 72, 3, 88
    x, res, dy, w, b = t(M, K), t(M, K), t(M, K), t(K), t(K)
    o = dict(a=e(M), q=e(M, K, dt=torch.int8), ra=e(M), ca=e(K), qr=e(M, K, dt=torch.int8), qc=e(K, M, dt=torch.int8), y=e(M, N, dt=BF),
             z=e(M, N, dt=BF), h=e(M, K, dt=BF), ly=e(M, K), mean=e(M), rstd=e(M), lq=e(M, K // 2, dt=torch.uint8),
             ls=e(M, -(-K // 16), dt=torch.uint8), la=e(M), dx=e(M, K, dt=BF), dw=e(K), db=e(K),
             kq=e(9, 8, H, D, dt=torch.int8), ka=e(9, 8, H), vq=e(9, 8, H, D, dt=torch.int8), va=e(9, 8, H), k2=e(M, H, D, dt=BF),
             v2=e(M, H, D, dt=BF))
    wq, wa = torch.randint(-127, 128, (N, K), generator=g).to(torch.int8).to(DEV), t(N, dt=FP).abs()
    bias, yres = t(N), t(M, N)
    k, v = t(M, H, D), t(M, 2 * H, D)[:, :H]
    table = torch.tensor([[4, 2, 0], [1, 3, 8]], dtype=torch.int32, device=DEV)
    starts, first = (torch.tensor(a, dtype=torch.int32, device=DEV) for a in ([0, 20, 35], [3, 7]))
    none = (None, None, None)
    torch.cuda.synchronize()
    s = dict(stream=stream)
    p.nvfp4_int8_quantize(x, o["a"], o["q"], **s)
    p.nvfp4_int8_quantize_rowcol(x, o["ra"], o["ca"], o["qr"], o["qc"], **s)
    p.nvfp4_int8_gemm(o["q"], LINE, o["a"], wq, LINE, wa, M, N, K, o["y"], bias=bias, act=p.NVFP4_ACT_SILU, residual=yres, z=o["z"], **s)
    p.nvfp4_layernorm(x, w, EPS, bias=b, residual=res, h=o["h"], y=o["ly"], mean=o["mean"], rstd=o["rstd"], q=o["lq"], s=o["ls"],
                      row_amax=o["la"], bound=448.0, **s)
    p.nvfp4_layernorm_backward(dy, o["h"], w, o["mean"], o["rstd"], o["dx"], dweight=o["dw"], dbias=o["db"], dres=res, **s)
    p.nvfp4_cache_write(k, v, o["kq"], None, o["ka"], o["vq"], None, o["va"], table, starts, first=first, **s)
    p.nvfp4_cache_read(o["k2"], o["v2"], o["kq"], None, o["ka"], o["vq"], None, o["va"], table, starts, first=first, **s)
    p.nvfp4_cache_write(k, None, o["kq"], None, o["ka"], *none, table, starts, **s)
    torch.cuda.synchronize()
    return o


def test_short_and_long_way_and_other_streams(monkeypatch):
    want = everything()
    assert not any(bool((t == 3).all()) for t in want.values())
    for stream in (torch.cuda.Stream(), None):
        for short in (p._short, Long()):
            monkeypatch.setattr(p, "_short", short)
            got = everything(stream)
            for n, t in want.items():
                assert torch.equal(t, got[n]), (n, stream, short)


def test_gradients_on_two_streams_at_once():
    """Each call's own workspace: sums of one do not reach the other's."""
    M, K = 3000, 2048
    g = torch.Generator().manual_seed(2)
    dy, h = (torch.randn(M, K, generator=g).to(BF).to(DEV) for _ in range(2))
    w = torch.ones(K, device=DEV)
    mean, rstd = torch.zeros(M, device=DEV), torch.ones(M, device=DEV)
    want = torch.empty(K, device=DEV), torch.empty(K, device=DEV)
    dx = torch.empty_like(dy)
    p.nvfp4_layernorm_backward(dy, h, w, mean, rstd, dx, dweight=want[0], dbias=want[1])
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [(torch.empty_like(dy), torch.empty(K, device=DEV), torch.empty(K, device=DEV)) for _ in range(12)]
    torch.cuda.synchronize()
    for i, (x, dw, db) in enumerate(outs):
        p.nvfp4_layernorm_backward(dy, h, w, mean, rstd, x, dweight=dw, dbias=db, stream=streams[i % 3])
    torch.cuda.synchronize()
    for x, dw, db in outs:
        assert torch.equal(x, dx) and torch.equal(dw, want[0]) and torch.equal(db, want[1])


def test_gradients_in_two_graphs():
    """Workspaces taken while capturing belong to their graph; replays by turns give what eager calls give."""
    K = 520
    w, graphs = torch.ones(K, device=DEV), []
    for M in (300, 900):
        t = [torch.zeros(M, K, device=DEV) for _ in range(3)] + [torch.zeros(M, device=DEV), torch.ones(M, device=DEV)]
        s = [torch.empty(K, device=DEV) for _ in range(2)]
        call = lambda t=t, s=s: p.nvfp4_layernorm_backward(t[0], t[1], w, t[3], t[4], t[2], dweight=s[0], dbias=s[1])
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append((t, s, call, graph))
    g = torch.Generator().manual_seed(3)
    for _ in range(4):
        want = []
        for t, s, call, _ in graphs:
            t[0].copy_(torch.randn(t[0].shape, generator=g))
            t[1].copy_(torch.randn(t[1].shape, generator=g))
            call()
            want.append([a.clone() for a in (t[2], *s)])
            for a in (t[2], *s):
                a.fill_(3)
        for *_, graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for (t, s, *_), e in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip((t[2], *s), e))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M,K", [(5, 8), (40, 9), (3, 263), (129, 255), (700, 1030), (2049, 513)])
def test_both_copies_of_a_view(M, K, dtype):
    """At odd addresses, the extreme element at either end of a line; NaN's amax is NaN, infinity's infinite."""
    g = torch.Generator().manual_seed(M + K)
    for shift in (1, 3):
        x = torch.empty(M * K + 8, dtype=dtype, device=DEV)[shift:shift + M * K].view(M, K)
        x.copy_(torch.randn(M, K, generator=g))
        x[0, K - 1] = 50
        x[M - 1, 0] = -60
        ra, ca = torch.full((M,), 3.0, device=DEV), torch.full((K,), 3.0, device=DEV)
        qr, qc = torch.empty(M, K, dtype=torch.int8, device=DEV), torch.empty(K, M, dtype=torch.int8, device=DEV)
        p.nvfp4_int8_quantize_rowcol(x, ra, ca, qr, qc)
        xf = x.float().cpu()
        assert torch.equal(ra.cpu(), xf.abs().amax(1)) and torch.equal(ca.cpu(), xf.abs().amax(0))
        assert torch.equal(qr.cpu(), codes(xf, xf.abs().amax(1, keepdim=True)))
        assert torch.equal(qc.cpu(), codes(xf, xf.abs().amax(0, keepdim=True)).t())
        x[M - 1, K - 1], x[0, 0] = float("nan"), float("-inf")
        p.nvfp4_int8_quantize_rowcol(x, ra, ca, qr, qc)
        ra, ca = ra.cpu(), ca.cpu()
        assert bool(ra[M - 1].isnan()) and bool(ca[K - 1].isnan()) and float(ra[0]) == float(ca[0]) == float("inf")
        assert torch.equal(ra[1:M - 1], xf.abs().amax(1)[1:M - 1])


# ------------------------------------------------------- past 32-bit offsets
def test_product_past_32_bits():
    """Lines of A, lines of B and outputs that lie past 2^32: each as a product of the last lines alone gives it."""
    say("[gpu] int8 product past 32 bits")
    K = 120000
    M = (1 << 32) // K + 300
    g = torch.Generator(device=DEV).manual_seed(1)
    A = torch.randint(-127, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
    B = torch.randint(-127, 128, (40, K), generator=g, device=DEV, dtype=torch.int8)
    aa, ab = torch.rand(M, device=DEV) + 0.5, torch.rand(40, device=DEV) + 0.5
    y, yt, part, part_t = (torch.empty(*s, device=DEV) for s in ((M, 40), (40, M), (100, 40), (40, 100)))
    p.nvfp4_int8_gemm(A, LINE, aa, B, LINE, ab, M, 40, K, y)
    p.nvfp4_int8_gemm(B, LINE, ab, A, LINE, aa, 40, M, K, yt)
    p.nvfp4_int8_gemm(A[-100:], LINE, aa[-100:], B, LINE, ab, 100, 40, K, part)
    p.nvfp4_int8_gemm(B, LINE, ab, A[-100:], LINE, aa[-100:], 40, 100, K, part_t)
    assert torch.equal(y[-100:], part) and torch.equal(yt[:, -100:], part_t)
    del A
    M = N = 66000
    A, B = (torch.randint(-127, 128, (M, 24), generator=g, device=DEV, dtype=torch.int8) for _ in range(2))
    aa, ab = torch.rand(M, device=DEV) + 0.5, torch.rand(N, device=DEV) + 0.5
    y, res = torch.full((M, N), 3, dtype=BF, device=DEV), torch.ones(M, N, dtype=BF, device=DEV)
    p.nvfp4_int8_gemm(A, LINE, aa, B, LINE, ab, M, N, 24, y, residual=res)
    part = torch.empty(77, N, dtype=BF, device=DEV)
    p.nvfp4_int8_gemm(A[-77:], LINE, aa[-77:], B, LINE, ab, 77, N, 24, part, residual=res[-77:])
    assert torch.equal(y[-77:], part)


def test_quantizers_past_32_bits():
    say("[gpu] int8 quantizers past 32 bits")
    M = K = 66000
    x = torch.ones(M, K, dtype=BF, device=DEV)
    g = torch.Generator().manual_seed(4)
    last, side = torch.randn(K, generator=g).to(BF), torch.randn(M, generator=g).to(BF)
    x[M - 1], x[:, K - 1] = last.to(DEV), side.to(DEV)
    ra, ca = torch.empty(M, device=DEV), torch.empty(K, device=DEV)
    qr, qc = torch.empty(M, K, dtype=torch.int8, device=DEV), torch.empty(K, M, dtype=torch.int8, device=DEV)
    p.nvfp4_int8_quantize_rowcol(x, ra, ca, qr, qc)
    row, col = x[M - 1:].float().cpu(), x[:, K - 1:].float().cpu()
    assert float(ra[M - 1]) == float(row.abs().max()) and float(ca[K - 1]) == float(col.abs().max())
    assert torch.equal(qr[M - 1:].cpu(), codes(row, row.abs().amax(1, keepdim=True)))
    assert torch.equal(qc[K - 1:].cpu().t(), codes(col, col.abs().amax(0, keepdim=True)))
    assert torch.equal(qr[:, K - 1:].cpu(), codes(col, ra.cpu()[:, None]))
    assert torch.equal(qc[:, M - 1:].cpu().t(), codes(row, ca.cpu()[None]))
    again = torch.full((M, K), 99, dtype=torch.int8, device=DEV)
    rb = torch.empty(M, device=DEV)
    p.nvfp4_int8_quantize(x, rb, again)
    assert torch.equal(ra, rb) and torch.equal(qr, again)


@pytest.mark.parametrize("M,K", [(1100000, 4000), (300000, 15000), (100000, 44000)])
def test_layer_norm_past_32_bits(M, K):
    """The last rows as calls on them alone give them; the sums of rows whose gradient is zero but for the last one's."""
    say(f"[gpu] layer norm past 32 bits {M}x{K}")
    assert M * K > 1 << 32
    x = torch.ones(M, K, dtype=BF, device=DEV)
    g = torch.Generator().manual_seed(5)
    tail = torch.randn(3, K, generator=g).to(BF).to(DEV)
    x[-3:] = tail
    w, b = torch.randn(K, generator=g).to(DEV), torch.randn(K, generator=g).to(DEV)

    def run(x):
        n = x.shape[0]
        o = dict(y=torch.empty_like(x), mean=torch.empty(n, device=DEV), rstd=torch.empty(n, device=DEV))
        p.nvfp4_layernorm(x, w, EPS, bias=b, **o)
        dy = o["y"]
        dy[:-1] = 0
        o["dx"], o["dw"], o["db"] = torch.empty_like(x), torch.empty(K, device=DEV), torch.empty(K, device=DEV)
        p.nvfp4_layernorm_backward(dy, x, w, o["mean"], o["rstd"], o["dx"], dweight=o["dw"], dbias=o["db"])
        return o
    one = run(tail)
    full = run(x)
    for n in ("y", "mean", "rstd", "dx"):
        assert torch.equal(full[n][-3:], one[n]), n
    assert torch.equal(full["dw"], one["dw"]) and torch.equal(full["db"], one["db"])
