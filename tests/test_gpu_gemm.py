"""The packed product against its definition in 64 bits.

Two kinds of operands. "Exact" ones, whose products are multiples of a quantum
so small in number that every FP32 sum is exact in any order: the output has
to equal the 64-bit one. Arbitrary ones, held to the bound of an FP32 sum:
with K terms in any order the error is at most K 2^-23 sum|u v| (2^-23, not
2^-24, so that adders which truncate are covered), and each later step adds a
rounding of its own.
"""
import numpy as np
import pytest
import torch

import precision_quantization_row_amd as p
from parity_utils import say
from product_utils import ACTS, DEV, E4M3, Lines, act64, np64, random_lines

pytestmark = pytest.mark.gpu
U = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    p.load_library()


def product(A, B, N, act="none", bias=None, residual=None, z=False, out=torch.float32, shift=0,
            stream=None, y=None, **kw):
    M, K = A.u.shape
    NB = 2 * N if act == "swiglu" else N
    a, sa, aa = A.dev(shift)
    b, sb, ab = B.dev(shift)
    y = torch.full((M, N), float("nan"), dtype=out, device=DEV) if y is None else y
    zt = torch.full((M, NB), float("nan"), dtype=out, device=DEV) if z else None
    torch.cuda.synchronize()
    p.nvfp4_gemm(a, sa, A.mode, aa, A.bound, b, sb, B.mode, ab, B.bound, M, N, K, y, bias=bias,
                 act=getattr(p, "NVFP4_ACT_" + act.upper()), residual=residual, z=zt, stream=stream, **kw)
    torch.cuda.synchronize()
    return y, zt


def z_and_bound(A, B):
    """The sum with its amax factors in 64 bits, and the bound of its FP32 error."""
    K = A.u.shape[1]
    f = A.line[:, None] * B.line[None, :]
    return A.u @ B.u.T * f, (K + 8) * U * (np.abs(A.u) @ np.abs(B.u).T * np.abs(f))


# one token to many, odd sizes, sizes around every tile and block edge
SHAPES = [(1, 1, 1), (1, 4096, 4096), (2, 17, 33), (3, 5, 15), (7, 130, 64), (16, 96, 1000), (17, 256, 128),
          (33, 64, 4097), (64, 64, 512), (65, 129, 257), (128, 128, 2048), (129, 300, 31), (130, 257, 16),
          (200, 515, 1111), (256, 256, 256), (257, 255, 640), (300, 1030, 96), (512, 512, 2880)]


@pytest.mark.parametrize("fmt", ["nvfp4", "e4m3"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_exact_sums(M, N, K, fmt):
    say(f"[gpu] gemm exact {M}x{N}x{K} {fmt}")
    rng = np.random.RandomState(M * 7 + N * 3 + K)
    A = random_lines(rng, M, K, fmt, exact=True)
    B = random_lines(rng, N, K, exact=True)
    y, _ = product(A, B, N)
    z = A.u @ B.u.T
    big = np.abs(A.u) @ np.abs(B.u).T * 4 < 2 ** 24   # exact in any order
    assert big.mean() > 0.999
    if fmt == "nvfp4":
        want = z * A.line[:, None] * B.line[None, :]
        assert np.array_equal(np64(y)[big], want[big])
    else:
        # RN(1/448) is no power of two: one rounding of the factor, one of the product
        want = z * A.line[:, None] * B.line[None, :]
        assert np.all(np.abs(np64(y) - want)[big] <= 3 * 2.0 ** -24 * np.abs(want)[big])


@pytest.mark.parametrize("fmt", ["nvfp4", "e4m3"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 72, 200), (5, 96, 64), (40, 66, 321), (130, 131, 96), (300, 260, 288)])
def test_epilogue(M, N, K, act, fmt):
    say(f"[gpu] gemm epilogue {M}x{N}x{K} {fmt} {act}")
    rng = np.random.RandomState(11 * M + K)
    NB = 2 * N if act == "swiglu" else N
    A = random_lines(rng, M, K, fmt)
    B = random_lines(rng, NB, K)
    z0, eb = z_and_bound(A, B)
    # bring z to the size activations see: an amax is a free factor
    A.amax = (A.amax / np.float32(np.sqrt(np.mean(z0 ** 2)))).astype(np.float32)
    A = Lines(A.q, A.s, A.amax, A.mode, A.bound, K)
    z0, eb = z_and_bound(A, B)
    for out, bdt in ((torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)):
        bias = torch.from_numpy(rng.standard_normal(NB).astype(np.float32)).to(DEV).to(bdt)
        res = torch.from_numpy(rng.standard_normal((M, N)).astype(np.float32)).to(DEV).to(out)
        z = z0 + np64(bias)
        zerr = eb + U * np.abs(z)
        half = 2.0 ** -24 if out == torch.float32 else 2.0 ** -8
        # slopes: gelu, silu below 1.2; relu2 2|z|; gated |up| and |gate| of the other half.
        # The sigmoid's exponential has relative error near |z| 2^-23
        y64 = act64(act, z, N)
        if act == "relu2":
            yerr = (2 * np.abs(z) + zerr) * zerr + 4 * U * np.abs(y64)
        elif act == "swiglu":
            g, u = z[:, :N], z[:, N:]
            silu = act64("silu", g, N)
            yerr = (1.2 * zerr[:, :N] + (4 + 4 * np.abs(g)) * U * np.abs(g)) * (np.abs(u) + zerr[:, N:]) \
                + np.abs(silu) * zerr[:, N:] + 4 * U * np.abs(y64)
        elif act == "none":
            yerr = zerr
        else:
            yerr = 1.2 * zerr + (8 + 8 * np.abs(z) + 2 * np.abs(z) ** 3) * U * np.abs(z)
        want = y64 + np64(res)
        y, zt = product(A, B, N, act, bias, res, True, out)
        # at most one rounding to the output's type
        assert np.all(np.abs(np64(zt) - z) <= zerr + half * (np.abs(z) + zerr))
        assert np.all(np.abs(np64(y) - want) <= yerr + 2 * U * np.abs(want) + half * (np.abs(want) + yerr))
        y2, _ = product(A, B, N, act, bias, res, False, out)   # without z: the same bits
        assert torch.equal(y, y2)


@pytest.mark.parametrize("am,bm", [(0, 0), (0, 1), (1, 0)])
@pytest.mark.parametrize("M", [1, 150])
def test_amax_modes_and_bounds(M, am, bm):
    rng = np.random.RandomState(5)
    A = random_lines(rng, M, 160, mode=am, bound=256.0)
    B = random_lines(rng, 70, 160, mode=bm, bound=448.0)
    z, e = z_and_bound(A, B)
    y, _ = product(A, B, 70)
    assert np.all(np.abs(np64(y) - z) <= e)


@pytest.mark.parametrize("shift", [1, 2, 4, 8, 12])
@pytest.mark.parametrize("fmt", ["nvfp4", "e4m3"])
@pytest.mark.parametrize("M", [3, 160])
def test_operands_at_any_address(M, fmt, shift):
    say(f"[gpu] gemm shift {shift} {M} {fmt}")
    rng = np.random.RandomState(shift)
    A = random_lines(rng, M, 256, fmt, exact=True)
    B = random_lines(rng, 130, 256, exact=True)
    want, _ = product(A, B, 130)
    got, _ = product(A, B, 130, shift=shift)
    assert torch.equal(want, got)


@pytest.mark.parametrize("M", [2, 140])
def test_outputs_at_any_address(M):
    """Outputs, residual and bias that start off every vector boundary."""
    rng = np.random.RandomState(2)
    N = 136
    A = random_lines(rng, M, 96, exact=True)
    B = random_lines(rng, N, 96, exact=True)
    for out in (torch.float32, torch.bfloat16):
        want, _ = product(A, B, N, out=out)
        buf = torch.zeros(M * N + 16, dtype=out, device=DEV)
        for s in (1, 2, 3, 5):
            buf.fill_(7.0)
            y = buf[s:s + M * N].view(M, N)
            product(A, B, N, out=out, y=y)
            assert torch.equal(y, want)
            assert torch.all(buf[:s] == 7.0) and torch.all(buf[s + M * N:] == 7.0)


def test_extreme_amaxes():
    """Factors whose product is ordinary but whose parts are not, and lines of
    zeros (amax 0)."""
    rng = np.random.RandomState(9)
    for M in (2, 140):
        A = random_lines(rng, M, 64, exact=True)
        B = random_lines(rng, 40, 64, exact=True)
        base = A.u @ B.u.T
        for ea, eb in ((100, -100), (-120, 110), (-130, 126), (118, -90)):
            A2 = Lines(A.q, A.s, np.full(M, 2.0 ** ea, np.float32), 1, A.bound, 64)
            B2 = Lines(B.q, B.s, np.full(40, 2.0 ** eb, np.float32), 1, B.bound, 64)
            y, _ = product(A2, B2, 40)
            assert np.array_equal(np64(y), base * 2.0 ** (ea + eb - 18))
        A2 = Lines(A.q, A.s, np.zeros(M, np.float32), 1, A.bound, 64)
        y, _ = product(A2, B, 40)
        assert torch.all(y == 0)


def test_garbage_outside_the_lines():
    """An odd line's spare nibble and the scales' neighbours are not read into
    the sum: two different paddings give the same bits."""
    rng = np.random.RandomState(4)
    for M, K in ((1, 33), (150, 33), (2, 4095), (140, 17)):
        A = random_lines(rng, M, K, exact=True)
        B = random_lines(rng, 50, K, exact=True)
        want, _ = product(A, B, 50)
        A.q[:, -1] |= 0x70
        B.q[:, -1] |= 0x50
        got, _ = product(A, B, 50)
        assert torch.equal(want, got)


@pytest.mark.parametrize("M", [4, 256])
def test_accumulates_in_place(M):
    """residual may be y's own buffer: adding to a main gradient."""
    rng = np.random.RandomState(8)
    A = random_lines(rng, M, 320, exact=True)
    B = random_lines(rng, 96, 320, exact=True)
    one, _ = product(A, B, 96)
    acc = torch.randn(M, 96, device=DEV)
    want = acc + one
    product(A, B, 96, residual=acc, y=acc)
    assert torch.equal(acc, want)


@pytest.mark.parametrize("M,N,K", [(1, 512, 8192), (130, 260, 4096), (48, 64, 28672)])
def test_same_bits_every_call_and_on_another_stream(M, N, K):
    rng = np.random.RandomState(6)
    A = random_lines(rng, M, K)
    B = random_lines(rng, N, K)
    first, _ = product(A, B, N)
    side = torch.cuda.Stream()
    for k in range(4):
        again, _ = product(A, B, N, stream=side if k % 2 else None)
        assert torch.equal(first, again)


def test_noop():
    rng = np.random.RandomState(1)
    for M in (1, 200):
        A = random_lines(rng, M, 64)
        B = random_lines(rng, 32, 64)
        y = torch.full((M, 32), 3.0, device=DEV)
        product(A, B, 32, y=y, noop=torch.ones(1, device=DEV))
        assert torch.all(y == 3.0)
        product(A, B, 32, y=y, noop=torch.zeros(1, device=DEV))
        assert not torch.any(y == 3.0)


@pytest.mark.parametrize("M", [2, 70])
def test_three_products_of_training(M):
    """Forward, data gradient and weight gradient from one matrix's two copies,
    against the dequantized operands."""
    N, K = 48, 80
    g = torch.Generator().manual_seed(3)
    mats = {n: torch.randn(*s, generator=g).to(DEV) for n, s in
            (("x", (M, K)), ("w", (N, K)), ("dy", (M, N)))}
    ops = {}
    for n, t in mats.items():
        R, C = t.shape
        o = p.empty_outputs(R, C, DEV)
        ra, ca = torch.empty(R, device=DEV), torch.empty(C, device=DEV)
        p.nvfp4_quantize_rowcol(t, ra, ca, 448.0, o["q_row"], o["s_row"], o["q_col"], o["s_col"])
        row, col = torch.empty(R, C, device=DEV), torch.empty(C, R, device=DEV)
        p.nvfp4_dequantize(o["q_row"], o["s_row"], R, C, 1, ra, 448.0, row)
        p.nvfp4_dequantize(o["q_col"], o["s_col"], C, R, 1, ca, 448.0, col)
        ops[n, "row"] = (o["q_row"], o["s_row"], ra, np64(row))
        ops[n, "col"] = (o["q_col"], o["s_col"], ca, np64(col))
    for (a, b, m, n, k) in ((("x", "row"), ("w", "row"), M, N, K), (("dy", "row"), ("w", "col"), M, K, N),
                            (("dy", "col"), ("x", "col"), N, K, M)):
        qa, sa, aa, va = ops[a]
        qb, sb, ab, vb = ops[b]
        y = torch.empty(m, n, device=DEV)
        p.nvfp4_gemm(qa, sa, 1, aa, 448.0, qb, sb, 1, ab, 448.0, m, n, k, y)
        # the dequantized values carry two roundings of their own each
        assert np.all(np.abs(np64(y) - va @ vb.T) <= (k + 12) * U * (np.abs(va) @ np.abs(vb).T))


def test_replays_in_a_graph():
    """A captured product, replayed on new inputs with eager work between, gives
    what the eager call gives."""
    rng = np.random.RandomState(12)
    for M, N, K in ((1, 256, 4096), (130, 128, 2048)):
        sets = [(random_lines(rng, M, K), random_lines(rng, N, K)) for _ in range(3)]
        a, sa, aa = sets[0][0].dev()
        b, sb, ab = sets[0][1].dev()
        y = torch.empty(M, N, device=DEV)
        call = lambda: p.nvfp4_gemm(a, sa, 1, aa, 448.0, b, sb, 1, ab, 448.0, M, N, K, y)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for A, B in sets + sets[:1]:
            want, _ = product(A, B, N)
            for t, v in ((a, A.dev()[0]), (sa, A.dev()[1]), (aa, A.dev()[2]), (b, B.dev()[0]), (sb, B.dev()[1]),
                         (ab, B.dev()[2])):
                t.copy_(v)
            y.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)


def test_refusals():
    rng = np.random.RandomState(1)
    A, B = random_lines(rng, 4, 32), random_lines(rng, 8, 32)
    a, sa, aa = A.dev()
    b, sb, ab = B.dev()
    y = torch.empty(4, 8, device=DEV)
    ok = dict(a=a, a_scale=sa, a_mode=1, a_amax=aa, a_bound=448.0, b=b, b_scale=sb, b_mode=1, b_amax=ab,
              b_bound=448.0, M=4, N=8, K=32, y=y)
    p.nvfp4_gemm(**ok)
    for bad in (dict(a=a.cpu()), dict(a_scale=None), dict(M=5), dict(N=9), dict(K=64), dict(a_amax=aa[:2]),
                dict(b=b.view(16, 8).t()), dict(residual=torch.empty(4, 7, device=DEV)),
                dict(bias=torch.empty(9, device=DEV)), dict(z=torch.empty(4, 16, device=DEV)),
                dict(act=p.NVFP4_ACT_SWIGLU)):
        with pytest.raises(ValueError):
            p.nvfp4_gemm(**{**ok, **bad})
    for bad in (dict(y=torch.empty(4, 8, device=DEV, dtype=torch.float16)), dict(b=b.float()),
                dict(residual=torch.empty(4, 8, device=DEV, dtype=torch.bfloat16)), dict(a=None),
                dict(bias=torch.empty(8, device=DEV, dtype=torch.float64))):
        with pytest.raises(TypeError):
            p.nvfp4_gemm(**{**ok, **bad})
    for bad, st in ((dict(a_bound=0.0), p.NVFP4_ERR_ARG), (dict(b_bound=449.0), p.NVFP4_ERR_ARG),
                    (dict(act=9), p.NVFP4_ERR_ARG), (dict(M=0, a=a[:0], a_scale=sa[:0], a_amax=aa[:0], y=y[:0]),
                                                     p.NVFP4_ERR_ARG)):
        with pytest.raises(p.Nvfp4Error) as e:
            p.nvfp4_gemm(**{**ok, **bad})
        assert e.value.status == st
    assert E4M3[8] == 2.0 ** -6
