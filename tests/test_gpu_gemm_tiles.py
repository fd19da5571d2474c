"""The packed product at sizes that take its large tiles, against its
definition in 64 bits on the GPU.

Operands are the exact ones of the small tests (every FP32 sum of their
products is exact in any order), so z without a bias has to be equal, a bias
costs one rounding, and y is held to the activation of the z that came back.
Which kernel a product takes goes by the times of both; tiles of 256 x 256 take
those with many lines and outputs, as here.
"""
import numpy as np
import pytest
import torch

import precision_quantization_row_amd as p
from parity_utils import say
from product_utils import DEV, random_lines

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    p.load_library()


def dev64(L):
    return torch.from_numpy(L.u).to(DEV), torch.from_numpy(np.array(L.line)).to(DEV)


def run(A, B, N, act="none", out=torch.float32, bias=None, residual=None, z=False, shift=0, noop=None):
    M, K = A.u.shape
    NB = 2 * N if act == "swiglu" else N
    a, sa, aa = A.dev(shift)
    b, sb, ab = B.dev(shift)
    y = torch.full((M, N), float("nan"), dtype=out, device=DEV)
    zt = torch.full((M, NB), float("nan"), dtype=out, device=DEV) if z else None
    p.nvfp4_gemm(a, sa, A.mode, aa, A.bound, b, sb, B.mode, ab, B.bound, M, N, K, y, bias=bias,
                 act=getattr(p, "NVFP4_ACT_" + act.upper()), residual=residual, z=zt, noop=noop)
    torch.cuda.synchronize()
    return y, zt


def exact_z(A, B):
    ua, la = dev64(A)
    ub, lb = dev64(B)
    big = torch.matmul(ua.abs(), ub.abs().t().contiguous()) * 4 < 2 ** 24
    assert big.double().mean() > 0.999
    return torch.matmul(ua, ub.t().contiguous()) * la[:, None] * lb[None, :], big


# ends of lines, tiles and stages: K around 16, 32, 64, 128 and their multiples
SHAPES = [(16385, 15400, 17), (12000, 11900, 31), (9000, 9010, 64), (8190, 8200, 65), (7000, 7010, 128),
          (6900, 7003, 129), (5000, 5001, 250), (4097, 4100, 385), (3700, 3600, 640), (2600, 4100, 1111), (300, 35000, 1500),
          (2049, 5121, 2047), (35000, 310, 1280)]


@pytest.mark.parametrize("fmt", ["nvfp4", "e4m3"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_exact_sums(M, N, K, fmt):
    say(f"[gpu] gemm tiles {M}x{N}x{K} {fmt}")
    rng = np.random.RandomState(M + N + K)
    A, B = random_lines(rng, M, K, fmt, exact=True), random_lines(rng, N, K, exact=True)
    y, _ = run(A, B, N)
    want, big = exact_z(A, B)
    if fmt == "nvfp4":
        assert torch.equal(y.double()[big], want[big])
    else:   # 1/448 is rounded once, the product once
        assert bool(((y.double() - want).abs() <= 3 * U * want.abs())[big].all())


@pytest.mark.parametrize("fmt", ["nvfp4", "e4m3"])
@pytest.mark.parametrize("act", ["none", "gelu", "silu", "relu2", "swiglu"])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_epilogue(act, fmt, out):
    say(f"[gpu] gemm tiles epilogue {act} {fmt} {out}")
    M, K = 2605, 400
    N = 3203 if act == "swiglu" else 6401
    NB = 2 * N if act == "swiglu" else N
    rng = np.random.RandomState(5)
    A, B = random_lines(rng, M, K, fmt, exact=True), random_lines(rng, NB, K, exact=True)
    g = torch.Generator().manual_seed(1)
    bias = torch.randn(NB, generator=g).to(DEV)
    res = torch.randn(M, N, generator=g).to(DEV).to(out)
    # bring z to the size activations see, by a power of two
    zz, _ = exact_z(A, B)
    A.amax = (A.amax * np.float32(2.0) ** -round(float(torch.log2(zz.std())))).astype(np.float32)
    A.line = A.amax.astype(np.float64) * (1 / 512.0 if fmt == "nvfp4" else np.float64(np.float32(1) / np.float32(448)))
    zz, big = exact_z(A, B)
    z64 = zz + bias.double()
    y, z = run(A, B, N, act, out, bias, res, True)
    # the factor's rounding and the product's (8-bit lines), then the bias's
    zerr = (0 if fmt == "nvfp4" else 3 * U) * zz.abs() + U * z64.abs()
    half = U if out == torch.float32 else 2.0 ** -8
    ok = (z.double() - z64).abs() <= zerr + half * (z64.abs() + zerr)
    assert bool(ok[big].all())
    a = z64.abs()
    if act == "none":
        want, err = z64, zerr
    elif act == "gelu":
        want = z64 * torch.sigmoid(2 * np.sqrt(2 / np.pi) * (z64 + 0.044715 * z64 ** 3))
        err = 1.2 * zerr + (16 + 16 * a + 4 * a ** 3) * U * a
    elif act == "silu":
        want, err = z64 * torch.sigmoid(z64), 1.2 * zerr + (16 + 16 * a) * U * a
    elif act == "relu2":
        want = z64.clamp(min=0) ** 2
        err = (2 * a + zerr) * zerr + 8 * U * want
    else:
        gate, up = z64[:, :N], z64[:, N:]
        silu = gate * torch.sigmoid(gate)
        want = silu * up
        err = (1.2 * zerr[:, :N] + (8 + 8 * gate.abs()) * U * gate.abs()) * (up.abs() + zerr[:, N:]) \
            + silu.abs() * zerr[:, N:] + 8 * U * want.abs()
        big = big[:, :N] & big[:, N:]
    want = want + res.double()
    ok = (y.double() - want).abs() <= err + 4 * U * want.abs() + half * (want.abs() + err)
    assert bool(ok[big].all())


def test_address_residual_in_place_and_noop():
    M, N, K = 2700, 4000, 512
    rng = np.random.RandomState(3)
    for fmt in ("nvfp4", "e4m3"):
        A, B = random_lines(rng, M, K, fmt, exact=True), random_lines(rng, N, K, exact=True)
        want, _ = run(A, B, N)
        for shift in (1, 4, 8):
            got, _ = run(A, B, N, shift=shift)
            assert torch.equal(want, got)
        y, _ = run(A, B, N, noop=torch.ones(1, device=DEV))
        assert bool(torch.isnan(y).all())
        acc = torch.randn(M, N, device=DEV)
        sum_ = acc + want
        a, sa, aa = A.dev()
        b, sb, ab = B.dev()
        p.nvfp4_gemm(a, sa, 1, aa, A.bound, b, sb, 1, ab, B.bound, M, N, K, acc, residual=acc)
        assert torch.equal(acc, sum_)


@pytest.mark.parametrize("M,N,K", [(4500000, 2, 16), (70000, 70, 33)])
def test_very_many_lines(M, N, K):
    """More workgroups along the lines than a grid's second axis holds."""
    say(f"[gpu] gemm tall {M}x{N}x{K}")
    rng = np.random.RandomState(9)
    A, B = random_lines(rng, M, K, exact=True), random_lines(rng, N, K, exact=True)
    y, _ = run(A, B, N)
    want, big = exact_z(A, B)
    assert torch.equal(y.double()[big], want[big])


def test_garbage_outside_odd_lines():
    M, N, K = 5000, 5001, 255
    rng = np.random.RandomState(4)
    A, B = random_lines(rng, M, K, exact=True), random_lines(rng, N, K, exact=True)
    want, _ = run(A, B, N)
    A.q[:, -1] |= 0x70
    B.q[:, -1] |= 0x50
    got, _ = run(A, B, N)
    assert torch.equal(want, got)


def test_same_bits_every_call():
    M, N, K = 2304, 4097, 8192
    rng = np.random.RandomState(6)
    A, B = random_lines(rng, M, K), random_lines(rng, N, K)
    first, _ = run(A, B, N)
    for _ in range(3):
        again, _ = run(A, B, N)
        assert torch.equal(first, again)
