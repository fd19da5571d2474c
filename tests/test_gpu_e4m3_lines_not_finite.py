"""E4M3 lines that hold a NaN or an infinity: every byte is a number, a zero in the cache (the line's amax carries what
the line holds), from every kernel that writes such lines; the lines beside them keep their bytes.
"""
import pytest
import torch

import precision_quantization_row_amd as p
from parity_utils import say
from product_utils import DEV
from test_gpu_int8_lines_not_finite import BF, BITS, FP, LENGTHS, lines

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    p.load_library()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("K", LENGTHS)
def test_norms(K, dtype):
    say(f"[gpu] norms of rows that are not finite {K} {dtype}")
    g = torch.Generator().manual_seed(K)
    M = 2 * len(BITS) + 1
    x, bad = lines(M, K, dtype, g)
    x, w = x.to(DEV), torch.randn(K, generator=g).to(DEV)
    for call in (p.nvfp4_layernorm, p.nvfp4_rmsnorm):
        amax, q = torch.empty(M, device=DEV), torch.full((M, K), 0x7F, dtype=torch.uint8, device=DEV)
        call(x, w, 1e-5, q=q.view(torch.float8_e4m3fn), row_amax=amax)
        assert bool(torch.isnan(amax.cpu()[bad]).all()) and not bool((q & 0x7F == 0x7F).any())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [7, 16, 100, 128, 256, 512, 1000, 1024])
def test_cache(D, dtype):
    say(f"[gpu] cached lines that are not finite {D} {dtype}")
    g = torch.Generator().manual_seed(D)
    T, H = 19, 2
    x, bad = lines(T * H, D, dtype, g)
    k, good = x.view(T, H, D).to(DEV), (~bad).view(T, H)
    table, starts = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.tensor([0, T], dtype=torch.int32, device=DEV)
    q, amax = torch.full((1, 32, H, D), 0x7F, dtype=torch.uint8, device=DEV), torch.zeros(1, 32, H, device=DEV)
    p.nvfp4_cache_write(k, None, q.view(torch.float8_e4m3fn), None, amax, None, None, None, table, starts)
    got = q[0, :T].cpu()
    assert not bool(got[~good].any())
    beside = x.float()[~bad]   # RN(x RN(448 / a)), to nearest even
    a = beside.abs().amax(1, keepdim=True)
    enc = torch.where(a > 0, torch.full_like(a, 448.0) / a, torch.ones_like(a))
    assert torch.equal(got[good], (beside * enc).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    out = torch.empty(T, H, D, device=DEV)
    p.nvfp4_cache_read(out, None, q.view(torch.float8_e4m3fn), None, amax, None, None, None, table, starts)
    fin = torch.isfinite(out.cpu())
    assert bool(fin[good].all()) and not bool(fin[~good].any())
