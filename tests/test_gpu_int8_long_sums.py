"""Sums of 2^17 products and more, past what a call takes: several calls on parts of the lines, y its own residual.

Tolerance: a part has 8 roundings of its own sum, U each, and each call but the first adds y, one more of the new sum.
"""
import pytest
import torch

import precision_quantization_row_amd as p
from parity_utils import say
from product_utils import DEV

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
LIMIT = (1 << 17) - 1


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    p.load_library()


@pytest.mark.parametrize("M,N", [(1, 40), (3, 33), (20, 64), (70, 130), (300, 600)])
@pytest.mark.parametrize("K", [LIMIT + 1, LIMIT + 6, 2 * LIMIT + 77])
def test_in_parts(M, N, K):
    say(f"[gpu] int8 product in parts {M}x{N}x{K}")
    g = torch.Generator().manual_seed(M + K)
    a, b = (torch.randint(-127, 128, (n, K), generator=g, dtype=torch.int8).to(DEV) for n in (M, N))
    aa, ab = torch.rand(M, generator=g).to(DEV) + 0.5, torch.rand(N, generator=g).to(DEV) + 0.5
    line, y = torch.full((M, N), float("nan"), device=DEV), torch.full((M, N), float("nan"), device=DEV)
    with pytest.raises(p.Nvfp4Error):
        p.nvfp4_int8_gemm(a, p.NVFP4_AMAX_LINE, aa, b, p.NVFP4_AMAX_LINE, ab, M, N, K, line)
    assert bool(torch.isnan(line).all())
    want, err = torch.zeros(M, N, dtype=torch.float64, device=DEV), torch.zeros(M, N, dtype=torch.float64, device=DEV)
    factor = (aa.double() / 127)[:, None] * (ab.double() / 127)[None]
    for k in range(0, K, LIMIT):
        n = min(LIMIT, K - k)
        qa, qb = a[:, k:k + n].contiguous(), b[:, k:k + n].contiguous()
        p.nvfp4_int8_gemm(qa, p.NVFP4_AMAX_LINE, aa, qb, p.NVFP4_AMAX_LINE, ab, M, N, n, y, residual=y if k else None)
        part = torch.matmul(qa.double(), qb.double().t().contiguous()) * factor
        err += 8 * U * part.abs()
        want += part
        if k:
            err += U * (want.abs() + err)
    assert bool(((y.double() - want).abs() <= err).all())
