"""The integer codes of lines that hold a NaN or an infinity: zeros, from every kernel that writes such lines; the lines
beside them keep their codes. NaNs of several signs and payloads: what their bits are must not show.
"""
import pytest
import torch

import precision_quantization_row_amd as p
from parity_utils import say
from product_utils import DEV
from test_gpu_int8 import codes

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
# FP32 patterns of NaNs (quiet and signalling, BF16 ones among them) and infinities
BITS = (0x7FC00000, -0x00400000, 0x7FFF0000, -0x00000001, 0x7F810000, 0x7FC12345, 0x7F800080, 0x7F800000, -0x00800000)
LENGTHS = [1, 7, 24, 100, 500, 513, 2000, 4000, 8000, 16001, 30000, 40000]   # each number of lanes a row takes


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    p.load_library()


def values(dtype):
    v = torch.tensor([b if b >= 0 else b + (1 << 32) for b in BITS], dtype=torch.int64)
    v = (v - (v >> 31 << 32)).to(torch.int32)
    if dtype == FP:
        return v.view(FP)
    top = (v >> 16).to(torch.int16)
    return top.view(BF)


def lines(M, K, dtype, g):
    """M rows, values(dtype)[i] somewhere in row 2 i + 1; (x, rows that hold one)."""
    x, v = torch.randn(M, K, generator=g).to(dtype), values(dtype)
    bits, vb = x.view(torch.int32 if dtype == FP else torch.int16), v.view(torch.int32 if dtype == FP else torch.int16)
    for i in range(len(v)):
        bits[2 * i + 1, int(torch.randint(0, K, (1,), generator=g))] = vb[i]
    bad = ~torch.isfinite(x.float()).all(1)
    return x, bad


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("K", LENGTHS)
def test_integer_rows(K, dtype):
    say(f"[gpu] rows that are not finite {K} {dtype}")
    g = torch.Generator().manual_seed(K)
    M = 2 * len(BITS) + 1
    x, bad = lines(M, K, dtype, g)
    assert int(bad.sum()) >= len(BITS) - 1   # (0x7F800080 is an infinity in BF16)
    amax, q = torch.empty(M, device=DEV), torch.full((M, K), 99, dtype=torch.int8, device=DEV)
    p.nvfp4_int8_quantize(x.to(DEV), amax, q)
    q, xf = q.cpu(), x.float()
    assert not bool(q[bad].any()) and not bool(torch.isfinite(amax.cpu()[bad]).any())
    assert torch.equal(q[~bad], codes(xf[~bad], xf[~bad].abs().amax(1, keepdim=True)))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M,K", [(19, 5), (19, 24), (130, 300), (300, 133), (200, 400), (256, 512)])
def test_integer_copies(M, K, dtype):
    say(f"[gpu] both copies, not finite {M}x{K} {dtype}")
    g = torch.Generator().manual_seed(M)
    x, bad = lines(M, K, dtype, g)
    xf = x.float()
    cbad = ~torch.isfinite(xf).all(0)
    ra, ca = torch.empty(M, device=DEV), torch.empty(K, device=DEV)
    qr, qc = torch.full((M, K), 99, dtype=torch.int8, device=DEV), torch.full((K, M), 99, dtype=torch.int8, device=DEV)
    p.nvfp4_int8_quantize_rowcol(x.to(DEV), ra, ca, qr, qc)
    qr, qc = qr.cpu(), qc.cpu()
    assert not bool(qr[bad].any()) and not bool(qc[cbad].any())
    assert torch.equal(qr[~bad], codes(xf[~bad], xf[~bad].abs().amax(1, keepdim=True)))
    good = xf[:, ~cbad]
    assert torch.equal(qc[~cbad], codes(good, good.abs().amax(0, keepdim=True)).t())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("K", LENGTHS)
def test_layer_norm(K, dtype):
    say(f"[gpu] layer norm of rows that are not finite {K} {dtype}")
    g = torch.Generator().manual_seed(K)
    M = 2 * len(BITS) + 1
    x, bad = lines(M, K, dtype, g)
    x, w = x.to(DEV), torch.randn(K, generator=g).to(DEV)
    amax, qi = torch.empty(M, device=DEV), torch.full((M, K), 99, dtype=torch.int8, device=DEV)
    p.nvfp4_layernorm(x, w, 1e-5, q=qi, row_amax=amax)
    assert bool(torch.isnan(amax.cpu()[bad]).all()) and not bool(qi.cpu()[bad].any())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [7, 16, 100, 128, 256, 512, 1000, 1024])
def test_cache(D, dtype):
    say(f"[gpu] cached lines that are not finite {D} {dtype}")
    g = torch.Generator().manual_seed(D)
    T, H = 19, 2
    x, bad = lines(T * H, D, dtype, g)
    k, good = x.view(T, H, D).to(DEV), (~bad).view(T, H)
    table, starts = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.tensor([0, T], dtype=torch.int32, device=DEV)
    q, amax = torch.full((1, 32, H, D), 99, dtype=torch.int8, device=DEV), torch.zeros(1, 32, H, device=DEV)
    p.nvfp4_cache_write(k, None, q, None, amax, None, None, None, table, starts)
    got = q[0, :T].cpu()
    assert not bool(got[~good].any())
    beside = x.float()[~bad]
    assert torch.equal(got[good], codes(beside, beside.abs().amax(1, keepdim=True)))
    out = torch.empty(T, H, D, device=DEV)
    p.nvfp4_cache_read(out, None, q, None, amax, None, None, None, table, starts)
    fin = torch.isfinite(out.cpu())
    assert bool(fin[good].all()) and not bool(fin[~good].any())
