"""The widest and tallest sizes. Every launch of the product, norm and gradient
calls at the largest sizes they accept: fewer than 2^32 threads, at most 65535
workgroups along y."""
import pytest

import launch_stub
import precision_quantization_row_amd as p
from launch_stub import act, gemm, norm, norm_bwd

COLS = 1 << 27
SIZES = [(1, COLS), (2, COLS), (2, COLS - 31), (2, COLS - 32), (255, COLS), (256, COLS), (300, COLS), (256, COLS - 2048),
         (1 << 30, 1), (1 << 30, 600), (1 << 26, 40000), (5, 32768), (1 << 20, 32769)]
CALLS = [f(M, K) for f in (norm, norm_bwd) for M, K in SIZES] + [norm_bwd(M, K, 1) for M, K in SIZES]
CALLS += [act(M, N, a) for M, N in SIZES for a in (1, 4)]
CALLS += [gemm(*s, act=a, fmt=f) for f in (1, 2) for a in (0, 4)
          for s in ((1, 1 << 26, 128), (1, (1 << 26) - 1, 1 << 23), (64, 1 << 22, 512), ((1 << 31) // 4, 1, 16), (1 << 20, 1 << 17, 64),
                    (1 << 22, 16, 1), (1 << 20, 64, 1 << 20), (17, 1 << 26, 64))]


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    return launch_stub.launches(CALLS, tmp_path_factory.mktemp("stub"))[1]


@pytest.mark.parametrize("i", range(len(CALLS)), ids=lambda i: f"{i}-{CALLS[i][0]}")
def test_threads_of_a_launch(launches, i):
    rc, grids = launches[i]
    assert rc == p.NVFP4_OK and grids, CALLS[i]
    for _, gx, gy, gz, bx, by, bz in grids:
        assert gz == by == bz == 1 and 1 <= bx <= 1024
        assert gx >= 1 and 1 <= gy <= 65535
        assert gx * gy * bx < 1 << 32, (CALLS[i], gx, gy, bx)


def test_the_stand_ins_see_the_launch(launches):
    """One row: one launch of one workgroup a row, so the grids above are real ones."""
    k = CALLS.index(norm(1, COLS))
    assert [g[1:] for g in launches[k][1]] == [[1, 1, 1, 1024, 1, 1]]


@pytest.mark.gpu
def test_widest_norm_gradient():
    """2^27 columns, the widest rows that are taken: the weight gradient of the
    first, the last and the middle columns, where its launches meet."""
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    dev, M, K = torch.device("cuda:0"), 2, COLS
    g = torch.Generator(device=dev).manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev, dtype=torch.bfloat16)
    dy, h, w = rand(M, K), rand(M, K), rand(K)
    r = torch.tensor([0.75, 1.25], device=dev)
    dx, dw = torch.full_like(dy, float("nan")), torch.full((K,), float("nan"), device=dev)
    p.nvfp4_rmsnorm_backward(dy, h, w, r, dx, dweight=dw)
    torch.cuda.synchronize()
    dot = [sum(float((dy[i, c:c + (1 << 24)].double() * w[c:c + (1 << 24)].double() * h[i, c:c + (1 << 24)].double()).sum())
               for c in range(0, K, 1 << 24)) for i in range(M)]
    for c in range(0, K, 1 << 24):
        s = slice(c, c + (1 << 24))
        d, x, xh = dy[:, s].double(), h[:, s].double(), h[:, s].double() * r.double()[:, None]
        # BF16 times 24 bits: one rounding in xh, one in each of the two sums' steps
        assert bool(((dw[s].double() - (d * xh).sum(0)).abs() <= 4 * 2.0 ** -24 * (d * xh).abs().sum(0)).all()), c
        mean = torch.tensor([dot[i] * float(r[i]) / K for i in range(M)], device=dev, dtype=torch.float64)
        want = r.double()[:, None] * (d * w[s].double() - xh * mean[:, None])
        # a lane's sum has K / 1024 = 2^17 terms: the mean is within 2^-7 of the terms' mean size, 0.51 r, and counts
        # r^2 |h| times; the output is rounded to BF16
        size = 2.0 ** -7 * 0.52 * r.double()[:, None] ** 3 * x.abs()
        assert bool(((dx[:, s].double() - want).abs() <= size + 2.0 ** -8 * (want.abs() + size) + 1e-6).all()), c
