"""The order in which the root-mean-square norm and its gradient join their sums: a lane's runs one after another, then
lanes 32, 16, 8, 4, 2 and 1 apart, then the waves in turn. A host that adds in that order gets the same bits.

Inputs are BF16 values, so that squares are exact; a fused step is then one rounding of a 64-bit sum that holds it
exactly (magnitudes from 2^-20 to 2^10 of 16-bit products, and a sum below 2^16).
"""
import numpy as np
import pytest
import torch

import precision_quantization_row_amd as p
from parity_utils import say
from product_utils import DEV

pytestmark = pytest.mark.gpu
f32 = np.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    p.load_library()


def joined(terms, threads):
    """FP32 sums [M] of float64 terms [M, K], each added to its lane's sum with one rounding."""
    M, K = terms.shape
    runs = -(-K // (8 * threads))
    t = np.zeros((M, runs * 8 * threads))
    t[:, :K] = terms
    t = t.reshape(M, runs, threads, 8)
    s = np.zeros((M, threads), f32)
    for j in range(runs):
        for k in range(8):
            s = (s + t[:, j, :, k]).astype(f32)
    s = s.reshape(M, threads // 64, 64)
    for o in (32, 16, 8, 4, 2, 1):
        s = s + s[:, :, np.arange(64) ^ o]
    out = s[:, 0, 0] if threads == 64 else np.zeros(M, f32)
    for w in range(threads // 64 if threads > 64 else 0):
        out = out + s[:, w, 0]
    return out


def inputs(M, K, g):
    x = torch.randn(M, K, generator=g).bfloat16().float()
    return torch.where(x.abs() < 2.0 ** -10, torch.full_like(x, 0.5), x)


# K, threads of a row's workgroup: the norm's, its gradient's
@pytest.mark.parametrize("K,forward,backward", [(40, 64, 64), (500, 64, 64), (2000, 256, 256), (2881, 256, 256), (4096, 256, 256),
                                                (8000, 1024, 512), (16384, 1024, 1024), (30000, 1024, 1024), (40000, 1024, 1024)])
def test_sums(K, forward, backward):
    say(f"[gpu] order of the norm's sums {K}")
    M, g = 48, torch.Generator().manual_seed(K)
    x, eps = inputs(M, K, g), f32(1e-5)
    want = f32(1) / np.sqrt(joined(x.double().numpy() ** 2, forward) / f32(K) + eps)
    for t in (x, x.bfloat16()):
        rstd = torch.empty(M, device=DEV)
        p.nvfp4_rmsnorm(t.to(DEV), torch.ones(K, device=DEV), float(eps), rstd=rstd)
        assert np.array_equal(rstd.cpu().numpy(), want)
    # gradient with r = 1: dot = sum dy h, dx = RN(dy - h mean)
    dy, one, dx = inputs(M, K, g), torch.ones(max(M, K), device=DEV), torch.empty(M, K, device=DEV)
    p.nvfp4_rmsnorm_backward(dy.to(DEV), x.to(DEV), one[:K], one[:M], dx)
    mean = joined(dy.double().numpy() * x.double().numpy(), backward) / f32(K)
    assert np.array_equal(dx.cpu().numpy(), (dy.double().numpy() - x.double().numpy() * mean[:, None].astype(np.float64)).astype(f32))
