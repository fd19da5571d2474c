"""The gradient of the product's epilogue against its formula in 64 bits and
against differences. The sigmoid's exponential has relative error near
|u| 2^-23 for argument u, and each step a rounding of 2^-24."""
import numpy as np
import pytest
import torch

import precision_quantization_row_amd as p
from parity_utils import say
from product_utils import ACTS, DEV, act64, dact64, np64

pytestmark = pytest.mark.gpu
U = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    p.load_library()


def code(act):
    return getattr(p, "NVFP4_ACT_" + act.upper())


def bound(act, dy, z, N):
    """|error| of the FP32 result: relative to the sizes of the terms."""
    a = np.abs(z)
    if act == "none":
        return 0 * dy
    if act == "relu2":
        return 2 * U * np.abs(dy) * 2 * a
    if act == "gelu":     # u = 2 sqrt(2/pi)(z + ..): |u| <= 1.6 |z| + 0.08 |z|^3; slope terms up to 1 + u' |z| / 4
        u = 1.6 * a + 0.08 * a ** 3
        return np.abs(dy) * (8 + 4 * u) * U * (1 + a * (1.6 + 0.22 * a * a) * np.minimum(0.25, np.exp(-np.minimum(u, 700))))
    if act == "silu":
        return np.abs(dy) * (8 + 4 * a) * U * (1 + a)
    g, u = a[:, :N], a[:, N:]
    return np.concatenate((np.abs(dy) * u * (8 + 4 * g) * U * (1 + g), np.abs(dy) * g * (8 + 4 * g) * U), 1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N", [(1, 1), (3, 7), (8, 16), (5, 2047), (9, 2056), (2, 4100), (4100, 24), (130, 515)])
def test_gradient(M, N, act, dtype):
    say(f"[gpu] act bwd {M}x{N} {act} {dtype}")
    rng = np.random.RandomState(M + N)
    NB = 2 * N if act == "swiglu" else N
    put = lambda a: torch.from_numpy(a.astype(np.float32)).to(DEV).to(dtype)
    dy, z = put(rng.standard_normal((M, N))), put(3 * rng.standard_normal((M, NB)))
    z[0, 0] = 0.0
    z[M // 2, NB - 1] = 60.0
    z[M - 1, NB // 2] = -60.0
    d64 = dact64(act, np64(dy), np64(z), N)
    e = bound(act, np64(dy), np64(z), N)
    dz, db = torch.full_like(z, float("nan")), torch.full((NB,), float("nan"), device=DEV)
    p.nvfp4_act_backward(dy, z, code(act), dz, dbias=db)
    torch.cuda.synchronize()
    half = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
    assert np.all(np.abs(np64(dz) - d64) <= e + half * (np.abs(d64) + e) + 1e-45)
    assert np.all(np.abs(np64(db) - d64.sum(0)) <= e.sum(0) + (M + 2) * U / 2 * (np.abs(d64) + e).sum(0) + 1e-45)
    dz2 = z.clone()
    p.nvfp4_act_backward(dy, dz2, code(act), dz2)   # in place, no bias
    assert torch.equal(dz2, dz)
    db2 = torch.empty_like(db)
    p.nvfp4_act_backward(dy, z, code(act), dz2, dbias=db2)
    assert torch.equal(db2, db)


@pytest.mark.parametrize("act", ACTS)
def test_differences(act):
    rng = np.random.RandomState(1)
    N = 50
    NB = 2 * N if act == "swiglu" else N
    z = (2 * rng.standard_normal((2, NB))).astype(np.float32).astype(np.float64)
    t = rng.standard_normal((2, N)).astype(np.float32).astype(np.float64)
    e = 1e-5
    want = np.empty_like(z)
    for i in range(2):
        for j in range(NB):
            d = np.zeros_like(z)
            d[i, j] = e
            want[i, j] = ((act64(act, z + d, N) - act64(act, z - d, N)) * t).sum() / (2 * e)
    f = lambda a: torch.from_numpy(a.astype(np.float32)).to(DEV)
    dz = torch.empty(2, NB, device=DEV)
    p.nvfp4_act_backward(f(t), f(z), code(act), dz)
    # relu2's second derivative jumps at 0: no z lies within e of it here
    assert np.abs(z).min() > 2 * e
    assert np.abs(np64(dz) - want).max() < 2e-5


def test_extremes():
    """Where exponentials overflow or vanish the gradients are their limits."""
    big = torch.tensor([[-3e38, -1e20, -200.0, -90.0, 90.0, 200.0, 1e18, 0.0]], device=DEV)
    one = torch.ones_like(big)
    for act, want in (("silu", [0, 0, 0, 0, 1, 1, 1, 0.5]), ("gelu", [0, 0, 0, 0, 1, 1, 1, 0.5])):
        dz = torch.empty_like(big)
        p.nvfp4_act_backward(one, big, code(act), dz)
        assert np.abs(np64(dz)[0] - np.array(want)).max() < 1e-6, act


@pytest.mark.parametrize("shift", [1, 2, 3])
def test_any_address(shift):
    for dtype in (torch.float32, torch.bfloat16):
        M, N = 5, 40
        mk = lambda n: torch.randn(n + 8, device=DEV).to(dtype)
        dy0, z0 = mk(M * N), mk(2 * M * N)
        dy, z = dy0[shift:shift + M * N].view(M, N), z0[shift:shift + 2 * M * N].view(M, 2 * N)
        want, got = torch.empty(M, 2 * N, dtype=dtype, device=DEV), mk(2 * M * N)
        p.nvfp4_act_backward(dy.clone(), z.clone(), code("swiglu"), want)
        v = got[shift:shift + 2 * M * N].view(M, 2 * N)
        p.nvfp4_act_backward(dy, z, code("swiglu"), v)
        assert torch.equal(v, want)


def test_noop_and_refusals():
    dy, z = torch.ones(4, 8, device=DEV), torch.ones(4, 16, device=DEV)
    dz, db = torch.full_like(z, 3.0), torch.full((16,), 3.0, device=DEV)
    p.nvfp4_act_backward(dy, z, code("swiglu"), dz, dbias=db, noop=torch.ones(1, device=DEV))
    assert torch.all(dz == 3.0) and torch.all(db == 3.0)
    with pytest.raises(ValueError):
        p.nvfp4_act_backward(dy, z, code("silu"), dz)
    with pytest.raises(ValueError):
        p.nvfp4_act_backward(dy, z, code("swiglu"), dz, dbias=db[:8])
    with pytest.raises(TypeError):
        p.nvfp4_act_backward(dy, z.bfloat16(), code("swiglu"), dz)
    with pytest.raises(p.Nvfp4Error):
        p.nvfp4_act_backward(dy, dy, 7, dy)
