"""The layer norm's gradient of rows of one value, so large that the mean times the deviation's reciprocal passes the
largest FP32 number: xh is 0 there and the gradient finite. Lanes past a row's end and row groups past the last row
have no elements: nothing of theirs may reach the sums.

Tolerances: a mean's terms pass at most depth(K) additions (a lane's share of the row, the tree over lanes and waves),
U of the magnitudes' sum each; xh, g and what joins them a handful of roundings; a column's sum passes M of them.
"""
import numpy as np
import pytest
import torch

import precision_quantization_row_amd as p
from parity_utils import say
from product_utils import DEV, np64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, FP = torch.bfloat16, torch.float32
# each number of lanes that a row takes, rows that are no multiple of a workgroup's, row ends inside a run and on one
SIZES = [(3, 5), (3, 7), (5, 96), (5, 100), (17, 128), (6, 500), (7, 512), (3, 2000), (3, 2047), (3, 2881), (2, 5000), (3, 8191),
         (2, 8200), (3, 16383), (2, 16400), (3, 17001), (300, 20)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    p.load_library()


def depth(K):
    return 8 * (K // 512 + 1) + 24


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M,K", SIZES)
def test_gradient(M, K, dtype):
    say(f"[gpu] layer norm gradient, large mean {M}x{K} {dtype}")
    g = torch.Generator().manual_seed(M + K)
    # sums of magnitudes have to stay below 2^128: of K times 2^121, K = 127 is the most
    for eps, top in ((1e-12, 2.0 ** 112), (1e-5, 2.0 ** 120 if K <= 127 else 2.0 ** 112)):
        h = torch.randn(M, K, generator=g) + 3
        h[1:] = top * torch.randint(1, 3, (M - 1, 1), generator=g)   # the last row among them
        h = h.to(dtype).to(DEV)
        w, b = torch.randn(K, generator=g).to(DEV), torch.randn(K, generator=g).to(DEV)
        dy, dres = (torch.randn(M, K, generator=g).to(dtype).to(DEV) for _ in range(2))
        y, mu, r = torch.empty(M, K, device=DEV), torch.empty(M, device=DEV), torch.empty(M, device=DEV)
        p.nvfp4_layernorm(h, w, eps, bias=b, y=y, mean=mu, rstd=r)
        assert torch.equal(mu[1:], h[1:, 0].float()) and torch.equal(y[1:], b.expand(M - 1, K))
        for d in (None, dres):
            dx, dw, db = torch.empty_like(dy), torch.empty(K, device=DEV), torch.empty(K, device=DEV)
            p.nvfp4_layernorm_backward(dy, h, w, mu, r, dx, dweight=dw, dbias=db, dres=d)
            h64, mu64, r64, g64 = np64(h), np64(mu)[:, None], np64(r)[:, None], np64(dy) * np64(w)
            xh = (h64 - mu64) * r64
            assert not xh[1:].any()
            m1, m2 = g64.mean(1, keepdims=True), (g64 * xh).mean(1, keepdims=True)
            want = r64 * (g64 - m1 - xh * m2) + (0 if d is None else np64(d))
            err = r64 * ((depth(K) + 6) * U * (np.abs(g64).mean(1, keepdims=True) + np.abs(xh) * np.abs(g64 * xh).mean(1, keepdims=True))
                         + 4 * U * (np.abs(g64) + np.abs(m1) + np.abs(xh * m2))) + 2 * U * np.abs(want)
            half = U if dtype == FP else 2.0 ** -8
            assert np.all(np.abs(np64(dx) - want) <= err + half * (np.abs(want) + err))
            assert np.all(np.abs(np64(dw) - (np64(dy) * xh).sum(0)) <= (M + 6) * U * np.abs(np64(dy) * xh).sum(0) + 1e-45)
            assert np.all(np.abs(np64(db) - np64(dy).sum(0)) <= (M + 4) * U * np.abs(np64(dy)).sum(0) + 1e-45)
