"""The product's second-level factors over the whole range of bounds: any
0 < bound <= 448 is accepted, and 1 / (bound 6) of two operands may leave FP32
where their amaxes bring the product back.

Operands are the exact ones, so a result carries the roundings of its factors
alone: bound 6, its reciprocal and the amax's mantissa times it, for both
operands, their product, and the sum times that: 8 of 2^-24."""
import numpy as np
import pytest
import torch

import precision_quantization_row_amd as p
from product_utils import DEV, np64, random_lines

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    p.load_library()


def product(A, B, N, K, bounds, amaxes):
    M = A.u.shape[0]
    a, sa, _ = A.dev()
    b, sb, _ = B.dev()
    aa, ab = (torch.full((n,), v, dtype=torch.float32, device=DEV) for n, v in zip((M, N), amaxes))
    y = torch.full((M, N), float("nan"), device=DEV)
    p.nvfp4_gemm(a, sa, 1, aa, bounds[0], b, sb, 1, ab, bounds[1], M, N, K, y)
    return np64(y), np64(aa)[0], np64(ab)[0]


BOUNDS = [(448.0, 448.0), (1.0, 256.0), (1e-3, 1e-3), (1e-19, 1e-19), (1e-25, 1e-20), (1e-38, 448.0), (1e-38, 1e-38),
          (2.0 ** -130, 2.0 ** -130), (2.0 ** -140, 1.0)]


@pytest.mark.parametrize("M,N,K", [(3, 40, 160), (40, 70, 64), (2600, 4100, 96)])
def test_small_bounds(M, N, K):
    rng = np.random.RandomState(M)
    A, B = random_lines(rng, M, K, exact=True), random_lines(rng, N, K, exact=True)
    ua, ub = (torch.from_numpy(L.u).to(DEV) for L in (A, B))
    base = np64(torch.matmul(ua, ub.t().contiguous()))
    for ba, bb in BOUNDS:
        # amaxes that bring the values to the size of the codes' own
        y, aa, ab = product(A, B, N, K, (ba, bb), (ba * 5.0, bb * 7.0))
        fa, fb = (np.float64(np.float32(b)) * 6.0 for b in (ba, bb))
        want = base * (aa / fa) * (ab / fb)
        assert np.all(np.abs(y - want) <= 8 * U * np.abs(want)), (ba, bb)


@pytest.mark.parametrize("M,N", [(2, 50), (2600, 4100)])
def test_block_scales_that_vanish(M, N):
    """A bound below E4M3's smallest value leaves block scales of zero: so is the product."""
    rng = np.random.RandomState(7)
    K = 64
    A, B = random_lines(rng, M, K), random_lines(rng, N, K)
    A.s[:], B.s[:] = 0, 0
    y, _, _ = product(A, B, N, K, (1e-30, 1e-30), (3.0, 5.0))
    assert np.all(y == 0)
