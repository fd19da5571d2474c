"""The 8-bit integer product's kernels, each at sizes that its choice leads to, odd in every direction, against
64 bits: sums, bias, residual, z, the gated pair, operands and outputs at odd addresses.

Tolerances: the sum's 8 roundings (U each), the bias' one, the residual's one, a rounding to the output's type.
"""
import pytest
import torch

import precision_quantization_row_amd as p
from parity_utils import say
from product_utils import DEV
from test_gpu_int8 import BF, FP, U, Lines, product, rand, z64

pytestmark = pytest.mark.gpu

# (lines of A and of B of the tile) -> sizes
PLAIN = {(64, 128): [(1030, 515, 101), (700, 700, 515)], (128, 128): [(4099, 2601, 515), (4099, 2601, 528)],
         (256, 256): [(4099, 4101, 101), (4099, 4100, 304)]}
GATED = {(64, 128): [(1030, 300, 101), (300, 700, 112)], (128, 128): [(4099, 1403, 515), (2059, 2601, 720)],
         (256, 256): [(4099, 2051, 101), (3001, 2601, 144)]}
# one token to some dozens, lines of less than a run to many units, B that passes 128 MB
FEW = [(1, 37, 5), (2, 130, 1025), (3, 1000, 4097), (4, 17, 1023), (1, 5, 16), (1, 1100, 122017), (2, 1100, 122017), (4, 1100, 122017),
       (7, 1100, 122017), (16, 9000, 15001), (30, 1100, 122017), (50, 1100, 122017)]
FEW_GATED = [(1, 9, 100), (2, 131, 1030), (3, 77, 2049), (4, 16, 15), (1, 560, 122017), (2, 560, 122017), (4, 560, 122017),
             (7, 560, 122017), (30, 560, 122017), (50, 560, 122017)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    p.load_library()


@pytest.mark.parametrize("M,N,K", [s for sizes in PLAIN.values() for s in sizes] + FEW)
def test_plain(M, N, K):
    say(f"[gpu] int8 tiles {M}x{N}x{K}")
    g = torch.Generator().manual_seed(M + N + K)
    A, B = Lines(g, M, K), Lines(g, N, K)
    z0, e0 = z64(A, B)
    for out, half in ((FP, U), (BF, 2.0 ** -8)):
        bias, res = rand(g, N, dtype=out), 100 * torch.randn(M, N, device=DEV).to(out)
        z = z0 + bias.double()
        e = e0 + U * (z.abs() + e0)
        y, zt = product(A, B, N, "none", out, True, bias=bias, residual=res)
        assert bool(((zt.double() - z).abs() <= e + half * (z.abs() + e)).all())
        want = z + res.double()
        e = e + U * (want.abs() + e)
        assert bool(((y.double() - want).abs() <= e + half * (want.abs() + e)).all())


@pytest.mark.parametrize("M,N,K", [s for sizes in GATED.values() for s in sizes] + FEW_GATED)
def test_gated(M, N, K):
    say(f"[gpu] int8 tiles gated {M}x{N}x{K}")
    g = torch.Generator().manual_seed(M + N + K)
    A, B = Lines(g, M, K), Lines(g, 2 * N, K)
    A.amax = A.amax / z64(A, B)[0].square().mean().sqrt().float()
    z0, e0 = z64(A, B)
    for out, half in ((FP, U), (BF, 2.0 ** -8)):
        bias, res = rand(g, 2 * N, dtype=out), torch.randn(M, N, device=DEV).to(out)
        z = z0 + bias.double()
        e = e0 + U * (z.abs() + e0)
        y, zt = product(A, B, N, "swiglu", out, True, bias=bias, residual=res)
        assert bool(((zt.double() - z).abs() <= e + half * (z.abs() + e)).all())
        gate, up, eg, eu = z[:, :N], z[:, N:], e[:, :N], e[:, N:]
        silu = gate * torch.sigmoid(gate)
        # silu's slope is below 1.2; its exponential's relative error is near |gate| 2^-23, and four roundings follow
        ey = (1.2 * eg + (4 + 4 * gate.abs()) * 2 * U * gate.abs()) * (up.abs() + eu) + silu.abs() * eu + 8 * U * (silu * up).abs()
        want = silu * up + res.double()
        ey = ey + 4 * U * want.abs()
        assert bool(((y.double() - want).abs() <= ey + half * (want.abs() + ey)).all())
        y2, _ = product(A, B, N, "swiglu", out, False, bias=bias, residual=res)
        assert torch.equal(y, y2)


@pytest.mark.parametrize("M,N,K", [(1, 333, 1111), (2, 333, 1111), (4, 333, 1111), (9, 333, 1111), (1030, 515, 101), (4099, 2601, 515), (4099, 4100, 304)])
def test_any_address(M, N, K):
    g = torch.Generator().manual_seed(K)
    A, B = Lines(g, M, K), Lines(g, N, K)
    want, _ = product(A, B, N, out=BF)
    A2, B2 = Lines(g, M, K, shift=4), Lines(g, N, K, shift=7)
    A2.q.copy_(A.q)
    B2.q.copy_(B.q)
    A2.amax, B2.amax = A.amax, B.amax
    buf = torch.full((M * N + 16,), 7.0, dtype=BF, device=DEV)
    y = buf[3:3 + M * N].view(M, N)
    product(A2, B2, N, out=BF, y=y)
    assert torch.equal(y, want)
    assert bool((buf[:3] == 7.0).all()) and bool((buf[3 + M * N:] == 7.0).all())
    y32, _ = product(A2, B2, N)
    one = y32.clone()
    product(A2, B2, N, residual=y32, y=y32)   # a value twice: exact
    assert torch.equal(y32, 2 * one)
