"""The norm's 8-bit codes over a whole training batch, against the definition in
64 bits, and call against call.

A code is E4M3_RNE of v = y 448 / amax. y and amax carry the same 1 / rms, so
its error leaves v; what stays is a rounding each of h, h r and y, the same
three of amax's element, 448 / a and the product: 8 roundings, |error of v| <=
8.01 2^-24 |v|. The code is the nearest E4M3 value of that v, so its distance
from the exact v is at most the nearest value's plus twice the error: only an
element within the error of a tie may round the other way."""
import numpy as np
import pytest
import torch

import precision_quantization_row_amd as p
from parity_utils import say
from product_utils import DEV, E4M3

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    p.load_library()


@pytest.mark.parametrize("M,K,dtype,res", [(16384, 4096, torch.bfloat16, True), (4097, 2881, torch.float32, False),
                                           (300, 28672, torch.bfloat16, True), (70, 40001, torch.float32, True)])
def test_codes_of_a_batch(M, K, dtype, res):
    say(f"[gpu] norm codes {M}x{K} {dtype}")
    g = torch.Generator(device=DEV).manual_seed(M + K)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)
    x = (rand(M, K) * torch.pow(10.0, 2 * torch.rand(M, 1, generator=g, device=DEV) - 1)).to(dtype)
    r = rand(M, K).to(dtype) if res else None
    w = (1 + 0.1 * rand(K)).to(dtype)
    h, q = torch.empty_like(x), torch.empty(M, K, dtype=torch.float8_e4m3fn, device=DEV)
    amax, rstd = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    call = lambda *o: p.nvfp4_rmsnorm(x, w, EPS, residual=r, h=o[0], q=o[1], row_amax=o[2], rstd=o[3])
    call(h, q, amax, rstd)
    for _ in range(3):   # equal calls give equal bits
        again = tuple(torch.empty_like(t) for t in (h, q, amax, rstd))
        call(*again)
        for a, b in zip((h, q, amax, rstd), again):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    grid = torch.from_numpy(np.unique(E4M3[np.isfinite(E4M3)])).to(DEV)
    for i in range(0, M, 2048):
        s = slice(i, i + 2048)
        h64 = x[s].double() + (r[s].double() if res else 0)
        y64 = h64 * ((h64 * h64).sum(1, keepdim=True) / K + EPS) ** -0.5 * w.double()
        v = y64 * (448.0 / y64.abs().amax(1, keepdim=True))
        hi = torch.searchsorted(grid, v).clamp_(1, grid.numel() - 1)
        nearest = torch.minimum((grid[hi] - v).abs(), (grid[hi - 1] - v).abs())
        assert bool(((q[s].double() - v).abs() <= nearest + 2 * 8.01 * U * v.abs()).all())
