"""Infinities and NaN. They are outside the quantizer's contract; what the
product, the norm and the gradients do with them: an element, line or row that
the formula makes NaN or infinite comes out so, its neighbours keep their bits,
and nothing that is not finite turns into a number on the way through the
norm's codes and the product (the row's amax carries it)."""
import numpy as np
import pytest
import torch

import precision_quantization_row_amd as p
from product_utils import ACTS, DEV, act64, dact64, np64, random_lines

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    p.load_library()


def same_kind(got, want):
    """NaN where the formula has NaN, the same infinity where it is infinite, finite elsewhere."""
    return (np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got == np.inf, want == np.inf)
            and np.array_equal(got == -np.inf, want == -np.inf))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N", [(3, 40), (40, 72), (2600, 4100)])
def test_through_the_products_epilogue(M, N, act):
    rng = np.random.RandomState(M)
    K, NB = 64, 2 * N if act == "swiglu" else N
    A, B = random_lines(rng, M, K, exact=True), random_lines(rng, NB, K, exact=True)
    a, sa, aa = A.dev()
    b, sb, ab = B.dev()
    aa, ab = aa / 64, ab / 64
    bias, res = torch.randn(NB, device=DEV), torch.randn(M, N, device=DEV)

    def run(aa, bias, res):
        y, z = torch.empty(M, N, device=DEV), torch.empty(M, NB, device=DEV)
        p.nvfp4_gemm(a, sa, 1, aa, A.bound, b, sb, 1, ab, B.bound, M, N, K, y, bias=bias, residual=res, z=z,
                     act=getattr(p, "NVFP4_ACT_" + act.upper()))
        return y, z
    y0, z0 = run(aa, bias, res)
    # one line's amax, three outputs' biases, two elements of the residual
    aa2, bias2, res2 = aa.clone(), bias.clone(), res.clone()
    aa2[1] = NAN
    bias2[3], bias2[N // 2], bias2[N - 1] = INF, -INF, NAN
    res2[0, 5], res2[2, 6] = NAN, -INF
    y, z = run(aa2, bias2, res2)
    hit = torch.zeros(M, N, dtype=torch.bool, device=DEV)
    hit[1] = True
    hit[:, 3] = hit[:, N // 2] = hit[:, N - 1] = True
    assert torch.equal(z[:, :N][~hit], z0[:, :N][~hit])
    if NB > N:   # (biases of gate lines: the up lines but one keep theirs)
        keep = torch.arange(M, device=DEV) != 1
        assert torch.equal(z[keep, N:], z0[keep, N:])
    clean = ~hit
    clean[0, 5] = clean[2, 6] = False
    assert torch.equal(y[clean], y0[clean])
    with np.errstate(all="ignore"):
        zw = np64(z0) - np64(bias) + np64(bias2)
        zw[1] = np.nan
        assert same_kind(np64(z), zw)
        assert same_kind(np64(y), act64(act, zw, N) + np64(res2))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_activation_gradient(act, dtype):
    M, N = 70, 515
    NB = 2 * N if act == "swiglu" else N
    dy, z = torch.randn(M, N, device=DEV).to(dtype), torch.randn(M, NB, device=DEV).to(dtype)

    def run(dy, z):
        dz, db = torch.empty(M, NB, dtype=dtype, device=DEV), torch.empty(NB, device=DEV)
        p.nvfp4_act_backward(dy, z, getattr(p, "NVFP4_ACT_" + act.upper()), dz, dbias=db)
        return dz, db
    dz0, db0 = run(dy, z)
    dy2, z2 = dy.clone(), z.clone()
    dy2[1, 4], dy2[2, 5], z2[3, 6] = NAN, INF, NAN
    dz, db = run(dy2, z2)
    with np.errstate(all="ignore"):
        want = dact64(act, np64(dy2), np64(z2), N)
    if act == "none":
        want = np64(dy2)
    assert same_kind(np64(dz), want)
    keep = torch.ones(M, NB, dtype=torch.bool, device=DEV)
    cols = [4, 5, 6] + ([N + 4, N + 5, N + 6] if NB > N else [])
    for r, c in ((1, 4), (2, 5), (3, 6)):
        keep[r, c] = False
        if NB > N:
            keep[r, N + c] = False
    assert torch.equal(dz[keep], dz0[keep])
    ok = torch.ones(NB, dtype=torch.bool, device=DEV)
    ok[cols] = False
    assert torch.equal(db[ok], db0[ok])
    with np.errstate(all="ignore"):
        assert same_kind(np64(db), want.sum(0))


@pytest.mark.parametrize("K", [96, 2881, 8192, 28672, 40000])
@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4"])
def test_norm_into_the_product(K, fmt):
    M, N = 6, 48
    x, w = torch.randn(M, K, device=DEV), torch.randn(K, device=DEV)
    rng = np.random.RandomState(1)
    B = random_lines(rng, N, K, exact=True)
    b, sb, ab = B.dev()

    def run(x):
        o = dict(h=torch.empty_like(x), y=torch.empty_like(x), rstd=torch.empty(M, device=DEV), row_amax=torch.empty(M, device=DEV))
        if fmt == "e4m3":
            o["q"], o["s"] = torch.empty(M, K, dtype=torch.float8_e4m3fn, device=DEV), None
        else:
            o["q"] = torch.empty(M, (K + 1) // 2, dtype=torch.uint8, device=DEV)
            o["s"] = torch.empty(M, (K + 15) // 16, dtype=torch.uint8, device=DEV)
        p.nvfp4_rmsnorm(x, w, 1e-5, **o)
        out = torch.empty(M, N, device=DEV)
        p.nvfp4_gemm(o["q"], o["s"], 1, o["row_amax"], 448.0, b, sb, 1, ab, B.bound, M, N, K, out)
        return o, out
    o0, out0 = run(x)
    x2 = x.clone()
    x2[1, 7], x2[2, K - 1], x2[4, K // 2] = NAN, INF, -INF
    o, out = run(x2)
    good = [0, 3, 5]
    for k in ("h", "y", "rstd", "row_amax", "q", "s"):
        if o[k] is not None:
            assert torch.equal(o[k][good].view(torch.uint8), o0[k][good].view(torch.uint8)), k
    assert torch.equal(out[good], out0[good])
    for row in (1, 2, 4):   # an infinite element: 1 / rms is 0, and its own product NaN
        assert bool(torch.isnan(o["row_amax"][row])) and bool(torch.isnan(o["y"][row]).any())
        assert bool(torch.isnan(out[row]).all())


@pytest.mark.parametrize("K", [96, 2881, 8192, 9000, 28672, 40000])
def test_norm_gradient(K):
    M = 5
    dy, h, w = torch.randn(M, K, device=DEV), torch.randn(M, K, device=DEV), torch.randn(K, device=DEV)
    r = torch.rand(M, device=DEV) + 0.5

    def run(dy):
        dx, dw = torch.empty_like(dy), torch.empty(K, device=DEV)
        p.nvfp4_rmsnorm_backward(dy, h, w, r, dx, dweight=dw)
        return dx, dw
    dx0, dw0 = run(dy)
    dy2 = dy.clone()
    dy2[2, 5] = NAN
    dx, dw = run(dy2)
    good = [0, 1, 3, 4]
    assert torch.equal(dx[good], dx0[good]) and bool(torch.isnan(dx[2]).all())
    ok = torch.arange(K, device=DEV) != 5
    assert torch.equal(dw[ok], dw0[ok]) and bool(torch.isnan(dw[5]))
