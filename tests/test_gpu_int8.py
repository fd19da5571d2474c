"""Lines of 8-bit integers and their product, against the definitions in 64 bits.

Codes bit for bit: amax exactly, then two rounded FP32 steps that the host takes
alike. Sums exactly: they are integers. What follows a sum s: its conversion,
RN(1/127) twice, a mantissa product for each line and one for both, and the
product with s: 8 roundings, U each; then the bias and the epilogue's own.
"""
import math

import numpy as np
import pytest
import torch

import precision_quantization_row_amd as p
from parity_utils import say
from product_utils import ACTS, DEV, act64, np64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, FP = torch.bfloat16, torch.float32
LINE, TENSOR = p.NVFP4_AMAX_LINE, p.NVFP4_AMAX_TENSOR


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    p.load_library()


def codes(x, amax):
    """x float32 on the host, amax broadcast: numpy's division, product and rint are the correctly rounded ones."""
    x, a = x.numpy(), amax.numpy()
    with np.errstate(all="ignore"):
        s = np.where(a == 0, np.float32(1), np.minimum(np.float32(127) / a, np.finfo(np.float32).max)).astype(np.float32)
        return torch.from_numpy(np.clip(np.rint(x * s), -127, 127).astype(np.int8))


def rand(g, *shape, dtype=FP, shift=0):
    n = math.prod(shape)
    buf = torch.empty(n + 8, dtype=dtype, device=DEV)[shift:shift + n]
    buf.copy_(torch.randn(n, generator=g).to(dtype))
    return buf.view(*shape)


# ------------------------------------------------------------------ quantize
ROWS = [(1, 1), (3, 7), (17, 8), (5, 16), (33, 120), (9, 128), (7, 129), (5, 512), (3, 513), (2, 2048), (3, 2881), (2, 4096),
        (2, 4104), (2, 8192), (2, 8200), (1, 16384), (2, 16400), (1, 28672), (1, 32768), (2, 32769), (1, 50001), (300, 40)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M,K", ROWS)
def test_rows(M, K, dtype):
    say(f"[gpu] int8 rows {M}x{K} {dtype}")
    g = torch.Generator().manual_seed(M * 31 + K)
    for shift in (0, 3):
        x = rand(g, M, K, dtype=dtype, shift=shift)
        amax = torch.empty(M, device=DEV)
        buf = torch.full((M * K + 16,), 99, dtype=torch.int8, device=DEV)
        q = buf[shift:shift + M * K].view(M, K)
        p.nvfp4_int8_quantize(x, amax, q)
        torch.cuda.synchronize()
        xf = x.float().cpu()
        assert torch.equal(amax.cpu(), xf.abs().amax(1))
        assert torch.equal(q.cpu(), codes(xf, xf.abs().amax(1, keepdim=True)))
        assert bool((buf[:shift] == 99).all()) and bool((buf[shift + M * K:] == 99).all())


BOTH = [(1, 1), (1, 300), (300, 1), (5, 8), (16, 16), (127, 129), (128, 128), (129, 127), (130, 264), (257, 1000), (1000, 257), (37, 2881)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M,K", BOTH)
def test_both_copies(M, K, dtype):
    say(f"[gpu] int8 rowcol {M}x{K} {dtype}")
    g = torch.Generator().manual_seed(M * 31 + K)
    for shift in (0, 1):
        x = rand(g, M, K, dtype=dtype, shift=shift)
        ra, ca = torch.empty(M, device=DEV), torch.empty(K, device=DEV)
        buf = torch.full((2, M * K + 16), 99, dtype=torch.int8, device=DEV)
        qr, qc = buf[0, shift:shift + M * K].view(M, K), buf[1, shift:shift + M * K].view(K, M)
        p.nvfp4_int8_quantize_rowcol(x, ra, ca, qr, qc)
        torch.cuda.synchronize()
        xf = x.float().cpu()
        assert torch.equal(ra.cpu(), xf.abs().amax(1)) and torch.equal(ca.cpu(), xf.abs().amax(0))
        assert torch.equal(qr.cpu(), codes(xf, xf.abs().amax(1, keepdim=True)))
        assert torch.equal(qc.cpu(), codes(xf, xf.abs().amax(0, keepdim=True)).t())
        assert bool((buf[:, :shift] == 99).all()) and bool((buf[:, shift + M * K:] == 99).all())
        # the rowwise copy is the one-pass quantizer's
        a1, q1 = torch.empty(M, device=DEV), torch.empty(M, K, dtype=torch.int8, device=DEV)
        p.nvfp4_int8_quantize(x, a1, q1)
        assert torch.equal(a1, ra) and torch.equal(q1, qr)


def test_values_at_the_borders():
    """Ties, lines of zeros, signed zeros, subnormal and huge lines."""
    rows = [[127.0] + [k + 0.5 for k in range(-126, 126)], [0.0] * 253, [-0.0] * 253, [1e-45] * 253, [2.0 ** -126] + [1e-45] * 252,
            [3e38] + [-1e38] * 252, [-254.0] + [2.0 * k + 1 for k in range(252)], [1.0] + [2.0 ** -30] * 252]
    x = torch.tensor(rows)
    M, K = x.shape
    for K_ in (K, 8 * K):   # another kernel for the longer rows
        xx = x.repeat(1, K_ // K).contiguous()
        amax, q = torch.empty(M, device=DEV), torch.empty(M, K_, dtype=torch.int8, device=DEV)
        p.nvfp4_int8_quantize(xx.to(DEV), amax, q)
        assert torch.equal(amax.cpu(), xx.abs().amax(1))
        assert torch.equal(q.cpu(), codes(xx, xx.abs().amax(1, keepdim=True)))
        ra, ca = torch.empty(M, device=DEV), torch.empty(K_, device=DEV)
        qr, qc = torch.empty(M, K_, dtype=torch.int8, device=DEV), torch.empty(K_, M, dtype=torch.int8, device=DEV)
        p.nvfp4_int8_quantize_rowcol(xx.to(DEV), ra, ca, qr, qc)
        assert torch.equal(qr, q) and torch.equal(qc.cpu(), codes(xx, xx.abs().amax(0, keepdim=True)).t())


# ------------------------------------------------------------------- product
class Lines:
    def __init__(self, g, R, K, mode=LINE, lo=-127, hi=127, shift=0):
        buf = torch.empty(R * K + 64, dtype=torch.int8, device=DEV)[shift:shift + R * K]
        buf.copy_(torch.randint(lo, hi + 1, (R * K,), generator=g).to(torch.int8))
        self.q, self.mode = buf.view(R, K), mode
        self.amax = torch.exp(6 * torch.rand(R if mode == LINE else 1, generator=g) - 3).to(DEV)
        self.u = self.q.double()

    def line(self):
        return (self.amax.double() / 127).expand(self.q.shape[0])


def product(A, B, N, act="none", out=FP, z=False, y=None, **kw):
    M, K = A.q.shape
    NB = 2 * N if act == "swiglu" else N
    y = torch.full((M, N), float("nan"), dtype=out, device=DEV) if y is None else y
    zt = torch.full((M, NB), float("nan"), dtype=out, device=DEV) if z else None
    torch.cuda.synchronize()
    p.nvfp4_int8_gemm(A.q, A.mode, A.amax, B.q, B.mode, B.amax, M, N, K, y, act=getattr(p, "NVFP4_ACT_" + act.upper()), z=zt, **kw)
    torch.cuda.synchronize()
    return y, zt


def z64(A, B):
    """The scaled sum in 64 bits, and 8 roundings of it. (The sums themselves are exact in float64.)"""
    z = torch.matmul(A.u, B.u.t().contiguous()) * A.line()[:, None] * B.line()[None, :]
    return z, 8 * U * z.abs()


# one token to many, odd sizes, sizes around every tile edge, k of part of a unit to many stages
SHAPES = [(1, 1, 1), (1, 4096, 4096), (2, 17, 33), (3, 5, 15), (7, 130, 64), (16, 96, 1000), (17, 256, 128), (16, 9000, 1111),
          (33, 64, 4097), (64, 64, 512), (65, 129, 257), (128, 128, 2048), (129, 300, 31), (130, 257, 16), (200, 515, 1111),
          (256, 256, 256), (257, 255, 640), (300, 1030, 96), (512, 512, 2880), (2600, 2600, 129), (2600, 2600, 144), (2605, 3203, 513),
          (4097, 2880, 2881), (4096, 2816, 2816), (1000, 8192, 300), (20, 300, 100001)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_sums(M, N, K):
    say(f"[gpu] int8 gemm {M}x{N}x{K}")
    g = torch.Generator().manual_seed(M * 7 + N * 3 + K)
    A, B = Lines(g, M, K), Lines(g, N, K)
    z, e = z64(A, B)
    y, _ = product(A, B, N)
    assert bool(((y.double() - z).abs() <= e).all())
    y2, _ = product(A, B, N, out=BF)   # the same value, rounded once
    assert torch.equal(y2, y.to(BF))


@pytest.mark.parametrize("M,N", [(1, 40), (20, 64), (70, 130), (300, 600), (2600, 2600)])
def test_the_largest_sums(M, N):
    """Codes of -128 and 127 throughout, K at its limit: sums up to 2^31 - 2^14."""
    K = (1 << 17) - 1 if M < 2600 else 32768
    say(f"[gpu] int8 gemm largest {M}x{N}")
    g = torch.Generator().manual_seed(M)
    A, B = Lines(g, M, K), Lines(g, N, K)
    for a, b in ((-128, -128), (-128, 127), (127, 127)):
        A.q.fill_(a)
        B.q.fill_(b)
        z = (A.line()[:, None] * B.line()[None, :]) * (a * b * K)
        y, _ = product(A, B, N)
        assert bool(((y.double() - z).abs() <= 8 * U * z.abs()).all())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 72, 200), (5, 96, 64), (20, 33, 1000), (40, 66, 321), (130, 131, 96), (300, 260, 288),
                                   (2600, 1400, 288), (2600, 1403, 291)])
def test_epilogue(M, N, K, act):
    say(f"[gpu] int8 gemm epilogue {M}x{N}x{K} {act}")
    g = torch.Generator().manual_seed(11 * M + K)
    NB = 2 * N if act == "swiglu" else N
    A, B = Lines(g, M, K), Lines(g, NB, K)
    A.amax = A.amax / z64(A, B)[0].square().mean().sqrt().float()   # z of the size activations see
    for out, bdt in ((FP, BF), (BF, FP)):
        bias, res = rand(g, NB, dtype=bdt), rand(g, M, N, dtype=out)
        z0, eb = z64(A, B)
        z, eb = np64(z0 + bias.double()), np64(eb)
        zerr = eb + U * (np.abs(z) + eb)
        half = U if out == FP else 2.0 ** -8
        # slopes: gelu, silu below 1.2; relu2 2|z|; gated |up| and |gate| of the other half. The sigmoid's exponential
        # has relative error near |z| 2^-23, gelu's the cube's besides
        y64, V = act64(act, z, N), 2 * U
        if act == "relu2":
            yerr = (2 * np.abs(z) + zerr) * zerr + 4 * V * np.abs(y64)
        elif act == "swiglu":
            gate, up = z[:, :N], z[:, N:]
            silu = act64("silu", gate, N)
            yerr = (1.2 * zerr[:, :N] + (4 + 4 * np.abs(gate)) * V * np.abs(gate)) * (np.abs(up) + zerr[:, N:]) \
                + np.abs(silu) * zerr[:, N:] + 4 * V * np.abs(y64)
        elif act == "none":
            yerr = zerr
        else:
            yerr = 1.2 * zerr + (8 + 8 * np.abs(z) + 2 * np.abs(z) ** 3) * V * np.abs(z)
        want = y64 + np64(res)
        y, zt = product(A, B, N, act, out, True, bias=bias, residual=res)
        assert np.all(np.abs(np64(zt) - z) <= zerr + half * (np.abs(z) + zerr))
        assert np.all(np.abs(np64(y) - want) <= yerr + 2 * V * np.abs(want) + half * (np.abs(want) + yerr))
        y2, _ = product(A, B, N, act, out, False, bias=bias, residual=res)   # without z: the same bits
        assert torch.equal(y, y2)


@pytest.mark.parametrize("am,bm", [(TENSOR, TENSOR), (TENSOR, LINE), (LINE, TENSOR)])
@pytest.mark.parametrize("M,N,K", [(1, 70, 160), (150, 70, 160), (2600, 1400, 160)])
def test_one_amax_for_all_lines(M, N, K, am, bm):
    g = torch.Generator().manual_seed(5)
    A, B = Lines(g, M, K, am), Lines(g, N, K, bm)
    z, e = z64(A, B)
    y, _ = product(A, B, N)
    assert bool(((y.double() - z).abs() <= e).all())


@pytest.mark.parametrize("shift", [1, 2, 4, 8, 15, 16])
@pytest.mark.parametrize("M,N,K", [(3, 130, 256), (160, 130, 256), (2600, 1300, 256), (2600, 1300, 257)])
def test_operands_at_any_address(M, N, K, shift):
    say(f"[gpu] int8 gemm shift {shift} {M}x{N}x{K}")
    g = torch.Generator().manual_seed(3)
    A, B = Lines(g, M, K), Lines(g, N, K)
    want, _ = product(A, B, N)
    for sa, sb in ((shift, shift), (0, shift), (shift, 0)):
        A2, B2 = Lines(g, M, K, shift=sa), Lines(g, N, K, shift=sb)
        A2.q.copy_(A.q)
        B2.q.copy_(B.q)
        A2.amax, B2.amax = A.amax, B.amax
        got, _ = product(A2, B2, N)
        assert torch.equal(want, got)


@pytest.mark.parametrize("M,N,K", [(2, 136, 96), (140, 136, 96), (2600, 1304, 96)])
def test_outputs_at_any_address(M, N, K):
    g = torch.Generator().manual_seed(2)
    A, B = Lines(g, M, K), Lines(g, N, K)
    for out in (FP, BF):
        want, _ = product(A, B, N, out=out)
        buf = torch.zeros(M * N + 16, dtype=out, device=DEV)
        for s in (1, 2, 3, 5):
            buf.fill_(7.0)
            y = buf[s:s + M * N].view(M, N)
            product(A, B, N, out=out, y=y)
            assert torch.equal(y, want)
            assert bool((buf[:s] == 7.0).all()) and bool((buf[s + M * N:] == 7.0).all())


@pytest.mark.parametrize("M", [2, 140, 2600])
def test_extreme_amaxes(M):
    g = torch.Generator().manual_seed(9)
    N, K = 1300 if M == 2600 else 40, 64
    A, B = Lines(g, M, K), Lines(g, N, K)
    base = torch.matmul(A.u, B.u.t().contiguous()) / 127 ** 2
    for ea, eb in ((100, -100), (-120, 110), (-130, 126), (118, -90)):
        A.amax, B.amax = torch.full((M,), 2.0 ** ea, device=DEV), torch.full((N,), 2.0 ** eb, device=DEV)
        y, _ = product(A, B, N)
        want = base * 2.0 ** (ea + eb)
        assert bool(((y.double() - want).abs() <= 8 * U * want.abs()).all())
    A.amax, B.amax = torch.zeros(M, device=DEV), torch.ones(N, device=DEV)
    y, _ = product(A, B, N)
    assert bool((y == 0).all())


def test_garbage_outside_the_lines():
    """Bytes before and behind the operands do not reach the sums."""
    g = torch.Generator().manual_seed(4)
    for M, N, K in ((1, 50, 33), (150, 50, 33), (2, 50, 4095), (2600, 1300, 129), (2600, 1300, 112)):
        A, B = Lines(g, M, K), Lines(g, N, K)
        outs = []
        for fill in (0, 85, -1):
            ops = []
            for L in (A, B):
                R = L.q.shape[0]
                buf = torch.full((R * K + 1024,), fill, dtype=torch.int8, device=DEV)
                view = buf[512:512 + R * K].view(R, K)
                view.copy_(L.q)
                ops.append(view)
            y = torch.empty(M, N, device=DEV)
            p.nvfp4_int8_gemm(ops[0], LINE, A.amax, ops[1], LINE, B.amax, M, N, K, y)
            outs.append(y)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
        z, e = z64(A, B)
        assert bool(((outs[0].double() - z).abs() <= e).all())


@pytest.mark.parametrize("M,N", [(4, 96), (256, 96), (2600, 1300)])
def test_accumulates_in_place(M, N):
    """residual may be y's own buffer: adding to a main gradient, and a sum longer than K's limit in parts."""
    g = torch.Generator().manual_seed(8)
    A, B = Lines(g, M, 320), Lines(g, N, 320)
    one, _ = product(A, B, N)
    acc = torch.randn(M, N, device=DEV)
    want = acc + one
    product(A, B, N, residual=acc, y=acc)
    assert torch.equal(acc, want)


@pytest.mark.parametrize("M,N,K", [(1, 512, 8192), (130, 260, 4096), (48, 64, 28672), (2600, 2600, 1024)])
def test_same_bits_every_call_and_on_another_stream(M, N, K):
    g = torch.Generator().manual_seed(6)
    A, B = Lines(g, M, K), Lines(g, N, K)
    first, _ = product(A, B, N)
    side = torch.cuda.Stream()
    for k in range(4):
        again, _ = product(A, B, N, stream=side if k % 2 else None)
        assert torch.equal(first, again)


def test_infinities_and_nan():
    """A NaN or infinite amax makes its own line so and no other; a NaN element reaches all products of its row's codes."""
    g = torch.Generator().manual_seed(7)
    for M, N in ((3, 40), (40, 72), (2600, 1300)):
        A, B = Lines(g, M, 64), Lines(g, N, 64)
        want, _ = product(A, B, N)
        A.amax = A.amax.clone()
        A.amax[1] = float("nan")
        y, _ = product(A, B, N)
        keep = torch.arange(M, device=DEV) != 1
        assert torch.equal(y[keep], want[keep]) and bool(torch.isnan(y[1]).all())
    for K in (40, 512, 2881, 40000):
        x = torch.randn(5, K, device=DEV)
        x[1, K // 2], x[3, K - 1] = float("nan"), float("inf")
        amax, q = torch.empty(5, device=DEV), torch.empty(5, K, dtype=torch.int8, device=DEV)
        p.nvfp4_int8_quantize(x, amax, q)
        B = Lines(g, 16, K)
        y = torch.empty(5, 16, device=DEV)
        p.nvfp4_int8_gemm(q, LINE, amax, B.q, LINE, B.amax, 5, 16, K, y)
        assert bool(torch.isnan(amax[1])) and bool(torch.isinf(amax[3])) and bool(torch.isnan(y[1]).all())
        assert not bool(torch.isfinite(y[3]).any()) and bool(torch.isfinite(y[[0, 2, 4]]).all())


@pytest.mark.parametrize("M", [2, 70, 300])
def test_three_products_of_training(M):
    """Forward, data gradient and weight gradient from one matrix's two copies."""
    N, K = 48, 80
    g = torch.Generator().manual_seed(3)
    ops = {}
    for n, s in (("x", (M, K)), ("w", (N, K)), ("dy", (M, N))):
        t = rand(g, *s, dtype=BF)
        R, C = s
        ra, ca = torch.empty(R, device=DEV), torch.empty(C, device=DEV)
        qr, qc = torch.empty(R, C, dtype=torch.int8, device=DEV), torch.empty(C, R, dtype=torch.int8, device=DEV)
        p.nvfp4_int8_quantize_rowcol(t, ra, ca, qr, qc)
        # within half a step of what was quantized, and three roundings
        assert bool(((qr.double() * (ra.double() / 127)[:, None] - t.double()).abs() <= (0.5 + 400 * U) * ra[:, None] / 127).all())
        assert bool(((qc.double() * (ca.double() / 127)[:, None] - t.double().t()).abs() <= (0.5 + 400 * U) * ca[:, None] / 127).all())
        ops[n, "row"], ops[n, "col"] = (qr, ra), (qc, ca)
    for (a, b, m, n, k) in ((("x", "row"), ("w", "row"), M, N, K), (("dy", "row"), ("w", "col"), M, K, N),
                            (("dy", "col"), ("x", "col"), N, K, M)):
        (qa, aa), (qb, ab) = ops[a], ops[b]
        y = torch.empty(m, n, device=DEV)
        p.nvfp4_int8_gemm(qa, LINE, aa, qb, LINE, ab, m, n, k, y)
        va, vb = qa.double() * (aa.double() / 127)[:, None], (qb.double() * (ab.double() / 127)[:, None]).t().contiguous()
        want = torch.matmul(va, vb)
        # (the scaled values' 64-bit sums are rounded themselves, k + 4 times 2^-53 of the magnitudes' sum: all there is of
        # a sum whose integers cancel)
        assert bool(((y.double() - want).abs() <= 9 * U * want.abs() + (k + 4) * 2.0 ** -53 * torch.matmul(va.abs(), vb.abs())).all())


def test_noop_and_replays_in_a_graph():
    """Captured quantizers and products, replayed on new inputs with eager work between, give what eager calls give."""
    g = torch.Generator().manual_seed(12)
    for M, N, K in ((1, 256, 4096), (130, 128, 2048), (2600, 1300, 528)):
        x, w = rand(g, M, K, dtype=BF), rand(g, N, K, dtype=BF)
        o = dict(q=torch.empty(M, K, dtype=torch.int8, device=DEV), a=torch.empty(M, device=DEV),
                 wr=torch.empty(N, K, dtype=torch.int8, device=DEV), wc=torch.empty(K, N, dtype=torch.int8, device=DEV),
                 ra=torch.empty(N, device=DEV), ca=torch.empty(K, device=DEV), y=torch.empty(M, N, device=DEV))

        def call(noop=None, stream=None):
            p.nvfp4_int8_quantize(x, o["a"], o["q"], noop=noop, stream=stream)
            p.nvfp4_int8_quantize_rowcol(w, o["ra"], o["ca"], o["wr"], o["wc"], noop=noop, stream=stream)
            p.nvfp4_int8_gemm(o["q"], LINE, o["a"], o["wr"], LINE, o["ra"], M, N, K, o["y"], noop=noop, stream=stream)
        for t in o.values():
            t.fill_(3)
        call(noop=torch.ones(1, device=DEV))
        assert all(bool((t == 3).all()) for t in o.values())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        call(noop=torch.zeros(1, device=DEV), stream=side)
        torch.cuda.synchronize()
        assert not bool((o["y"] == 3).all())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for k in range(4):
            x.copy_(torch.randn(M, K, generator=g))
            w.copy_(torch.randn(N, K, generator=g))
            call()
            want = {n: t.clone() for n, t in o.items()}
            for t in o.values():
                t.fill_(3)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(t, want[n]) for n, t in o.items())


def test_refusals():
    g = torch.Generator().manual_seed(1)
    A, B = Lines(g, 4, 32), Lines(g, 8, 32)
    y = torch.empty(4, 8, device=DEV)
    ok = dict(a=A.q, a_mode=LINE, a_amax=A.amax, b=B.q, b_mode=LINE, b_amax=B.amax, M=4, N=8, K=32, y=y)
    p.nvfp4_int8_gemm(**ok)
    for bad in (dict(a=A.q.cpu()), dict(M=5), dict(N=9), dict(K=64), dict(a_amax=A.amax[:2]), dict(b=B.q.t()),
                dict(residual=torch.empty(4, 7, device=DEV)), dict(bias=torch.empty(9, device=DEV)),
                dict(z=torch.empty(4, 16, device=DEV)), dict(act=p.NVFP4_ACT_SWIGLU)):
        with pytest.raises(ValueError):
            p.nvfp4_int8_gemm(**{**ok, **bad})
    for bad in (dict(y=torch.empty(4, 8, device=DEV, dtype=torch.float16)), dict(b=B.q.float()), dict(a=None),
                dict(a=A.q.view(torch.uint8)), dict(residual=torch.empty(4, 8, device=DEV, dtype=BF)),
                dict(bias=torch.empty(8, device=DEV, dtype=torch.float64))):
        with pytest.raises((TypeError, ValueError)):
            p.nvfp4_int8_gemm(**{**ok, **bad})
    for bad in (dict(act=9), dict(b=None), dict(b_amax=None)):
        with pytest.raises(p.Nvfp4Error):
            p.nvfp4_int8_gemm(**{**ok, **bad})
    x, a, q = torch.zeros(4, 32, device=DEV), torch.empty(4, device=DEV), torch.empty(4, 32, dtype=torch.int8, device=DEV)
    for bad in ((x, a[:3], q), (x, a, q[:3]), (x.view(2, 2, 32), a, q), (x.t(), a, q)):
        with pytest.raises(ValueError):
            p.nvfp4_int8_quantize(*bad)
    for bad in ((x.half(), a, q), (x, a, q.view(torch.uint8)), (x, a.double(), q)):
        with pytest.raises(TypeError):
            p.nvfp4_int8_quantize(*bad)
    with pytest.raises(ValueError):
        p.nvfp4_int8_quantize_rowcol(x, a, a, q, q)
