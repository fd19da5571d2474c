"""Every kernel of the product, the norm and the gradients at sizes that give its
loops several turns, against 64-bit forms on the GPU; and, on the host, that
these sizes reach every one of them.

The product's operands are exact ones (block scales 1 .. 8, 8-bit values of
whole numbers, amaxes powers of two): every FP32 sum of their products is exact
in any order, so z has to be equal (8-bit lines: within three roundings, since
1 / 448 is no power of two)."""
import math

import pytest
import torch

import launch_stub
import precision_quantization_row_amd as p
from parity_utils import say
from product_utils import ACTS
from variant_cases import ACT, GATED, GEMM, NORM, NORM_BWD

U = 2.0 ** -24
BF, FP = torch.bfloat16, torch.float32
TYPES = [(BF, BF), (FP, FP), (BF, FP), (FP, BF)]


def _dev():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    return torch.device("cuda:0")


def test_sizes_reach_every_kernel(tmp_path):
    calls = [launch_stub.gemm(*s, fmt=f) for s in GEMM for f in (1, 2)]
    calls += [launch_stub.gemm(*s, act=p.NVFP4_ACT_SWIGLU, fmt=f) for s in GATED for f in (1, 2)]
    calls += [f(*s, dt, wd) for f, sizes in ((launch_stub.norm, NORM), (launch_stub.norm_bwd, NORM_BWD)) for s in sizes
              for dt in (0, 1) for wd in (0, 1)]
    calls += [launch_stub.act(*s, a, dt) for s in ACT for a in range(5) for dt in (0, 1)]
    names, out = launch_stub.launches(calls, tmp_path)
    assert all(rc == p.NVFP4_OK for rc, _ in out)
    # (a name starts with its length in the mangled form: 5nvfp416gemm_rows_kernel..)
    ours = {n for n in names if any(k in n for k in ("gemm_", "norm_", "act_bwd", "colsum"))}
    assert len(ours) > 60
    assert not ours - {launch[0] for _, grids in out for launch in grids}
    # more rows than workgroups in every kernel of the norm's gradient
    for call, (_, grids) in zip(calls, out):
        if call[0] == "nvfp4_rmsnorm_backward":
            assert call[2][7] > max(g[1] for g in grids if "norm_bwd" in g[0])


# ------------------------------------------------------------------- product
E2M1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
BOUND = 512.0 / 6.0   # FP32: 1 / (bound 6) is 2^-9


def exact_lines(g, R, K, fmt, dev):
    """(codes, block scales, amaxes, values in 64 bits without amaxes, factors in 64 bits)"""
    rnd = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=dev)
    amax = torch.pow(2.0, rnd(-3, 4, R).float())
    if fmt == "e4m3":
        u = (rnd(1, 9, R, K) * (2 * rnd(0, 2, R, K) - 1)).float()
        return u.to(torch.float8_e4m3fn), None, amax * 448, u.double(), (amax * 448).double() * float(torch.tensor(1.0) / 448)
    q, s = rnd(0, 256, R, (K + 1) // 2).to(torch.uint8), rnd(1, 9, R, (K + 15) // 16).float()
    lut = torch.tensor(E2M1 + [-v for v in E2M1], device=dev, dtype=torch.float64)
    u = torch.stack((lut[(q & 15).int()], lut[(q >> 4).int()]), 2).view(R, -1)[:, :K]   # (an odd line's last nibble: garbage)
    u = u * s.double().repeat_interleave(16, 1)[:, :K]
    return q, s.to(torch.float8_e4m3fn), amax, u, amax.double() / 512


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "e4m3"])
@pytest.mark.parametrize("gated,M,N,K", [(0, *s) for s in GEMM] + [(1, *s) for s in GATED])
def test_product(gated, M, N, K, fmt):
    dev = _dev()
    say(f"[gpu] variants: product {M}x{N}x{K} {fmt} gated {gated}")
    g = torch.Generator(device=dev).manual_seed(M * 7 + N * 3 + K + gated)
    NB = 2 * N if gated else N
    qa, sa, aa, ua, fa = exact_lines(g, M, K, fmt, dev)
    qb, sb, ab, ub, fb = exact_lines(g, NB, K, "nvfp4", dev)
    # gated: z near 1, by a power of two
    size = 2.0 ** -round(math.log2(math.sqrt(K) * 150 / 512 * (1 if fmt == "e4m3" else 1 / 256))) if gated else 1.0
    aa, fa = aa * size, fa * size
    y, z = torch.full((M, N), float("nan"), device=dev), torch.full((M, NB), float("nan"), device=dev)
    torch.cuda.synchronize()
    p.nvfp4_gemm(qa, sa, 1, aa, BOUND, qb, sb, 1, ab, BOUND, M, N, K, y, z=z,
                 act=p.NVFP4_ACT_SWIGLU if gated else p.NVFP4_ACT_NONE)
    torch.cuda.synchronize()
    ubt = ub.t().contiguous()
    big = torch.matmul(ua.abs(), ubt.abs()) * 4 < 2 ** 24
    assert float(big.double().mean()) > 0.999
    want = torch.matmul(ua, ubt) * fa[:, None] * fb[None, :]
    if fmt == "nvfp4":
        assert torch.equal(z.double()[big], want[big])
    else:
        assert bool(((z.double() - want).abs() <= 3 * U * want.abs())[big].all())
    assert not bool(torch.isnan(z).any())
    if not gated:
        assert torch.equal(y, z)
        return
    # y from the z that came back; the sigmoid's error is near |gate| + 8 roundings, and it may vanish below FP32's smallest
    gate, up = z[:, :N].double(), z[:, N:].double()
    ref = gate * torch.sigmoid(gate) * up
    assert bool(((y.double() - ref).abs() <= (16 + 4 * gate.abs()) * U * ref.abs() + 1e-34 * (1 + up.abs())).all())
    assert float(z.std()) < 100   # (so that the gates say something)


# -------------------------------------------------------------- norm, backward
def depth(K):
    """Additions that a term of a row's sum passes: a lane's share of it, then lanes and waves."""
    return 8 * (K // 512 + 1) + 24


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,wdtype", TYPES)
@pytest.mark.parametrize("M,K", NORM_BWD)
def test_norm_backward(M, K, dtype, wdtype):
    dev = _dev()
    say(f"[gpu] variants: norm gradient {M}x{K} {dtype} {wdtype}")
    g = torch.Generator(device=dev).manual_seed(M + K)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)
    dy, h, dres, w = rand(M, K).to(dtype), rand(M, K).to(dtype), rand(M, K).to(dtype), rand(K).to(wdtype)
    r = torch.rsqrt(h.float().square().mean(1) + 1e-5)
    r64, half = r.double()[:, None], U if dtype == FP else 2.0 ** -8
    xh, gg = h.double() * r64, dy.double() * w.double()
    dw64, dwsum = (dy.double() * xh).sum(0), (dy.double() * xh).abs().sum(0)
    base = r64 * (gg - xh * (gg * xh).mean(1, keepdim=True))
    # the mean's terms pass depth(K) additions; then a handful of roundings
    err = r64 * ((depth(K) + 6) * U * xh.abs() * (gg * xh).abs().mean(1, keepdim=True) + 4 * U * gg.abs())
    for d in (None, dres):
        want = base if d is None else base + d.double()
        e = err + 2 * U * want.abs()
        dx, dw = torch.full_like(dy, float("nan")), torch.full((K,), float("nan"), device=dev)
        p.nvfp4_rmsnorm_backward(dy, h, w, r, dx, dweight=dw, dres=d)
        torch.cuda.synchronize()
        assert bool(((dx.double() - want).abs() <= e + half * (want.abs() + e)).all())
        assert bool(((dw.double() - dw64).abs() <= (M + 4) * U * dwsum).all())
        dx2, dw2 = torch.empty_like(dx), torch.empty_like(dw)
        p.nvfp4_rmsnorm_backward(dy, h, w, r, dx2, dres=d)      # without the weight's gradient: the same bits
        assert torch.equal(dx, dx2)
        at = dy.clone() if d is None else d.clone()             # dx over dy, or over dres
        p.nvfp4_rmsnorm_backward(at if d is None else dy, h, w, r, at, dweight=dw2, dres=None if d is None else at)
        assert torch.equal(at, dx) and torch.equal(dw2, dw)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M,K", [(1, 24), (5, 513), (5, 2880), (5, 9000), (3, 28000), (3, 40000)])
def test_norm_backward_at_any_address(M, K, dtype):
    dev = _dev()
    g = torch.Generator(device=dev).manual_seed(K)
    for shift in (1, 2, 3):
        def at(*s, dt=dtype):
            n = math.prod(s)
            buf = torch.full((n + 8,), 5.0, device=dev, dtype=dt)
            buf[shift:shift + n] = torch.randn(n, generator=g, device=dev).to(dt)
            return buf, buf[shift:shift + n].view(*s)
        (_, dy), (_, h), (_, dres), (_, w), (_, r) = at(M, K), at(M, K), at(M, K), at(K), at(M, dt=FP)
        (bx, dx), (bw, dw) = at(M, K), at(K, dt=FP)
        want, wantw = torch.empty(M, K, device=dev, dtype=dtype), torch.empty(K, device=dev)
        p.nvfp4_rmsnorm_backward(dy.clone(), h.clone(), w.clone(), r.clone(), want, dweight=wantw, dres=dres.clone())
        p.nvfp4_rmsnorm_backward(dy, h, w, r, dx, dweight=dw, dres=dres)
        assert torch.equal(dx, want) and torch.equal(dw, wantw)
        for buf in (bx, bw):
            n = buf.numel() - 8
            assert bool((buf[:shift] == 5.0).all()) and bool((buf[shift + n:] == 5.0).all())


# --------------------------------------------------------------- norm, forward
@pytest.mark.gpu
@pytest.mark.parametrize("dtype,wdtype", TYPES)
@pytest.mark.parametrize("M,K", NORM)
def test_norm(M, K, dtype, wdtype):
    dev = _dev()
    g = torch.Generator(device=dev).manual_seed(M + K)
    x, w = torch.randn(M, K, generator=g, device=dev).to(dtype), torch.randn(K, generator=g, device=dev).to(wdtype)
    y, rstd = torch.empty(M, K, device=dev), torch.empty(M, device=dev)
    p.nvfp4_rmsnorm(x, w, 1e-5, y=y, rstd=rstd)
    r64 = (x.double().square().mean(1) + 1e-5) ** -0.5
    rel = (depth(K) / 2 + 8) * U
    assert bool(((rstd.double() - r64).abs() <= rel * r64).all())
    want = x.double() * r64[:, None] * w.double()
    assert bool(((y.double() - want).abs() <= (rel + 4 * U) * want.abs()).all())


@pytest.mark.gpu
def test_norm_of_more_rows_than_a_launch_holds():
    """2^20 rows a launch: the ones after it, and the ones before, as calls of their own give them."""
    dev, M, K = _dev(), (1 << 20) + 5, 40
    g = torch.Generator(device=dev).manual_seed(1)
    x, w = torch.randn(M, K, generator=g, device=dev), torch.randn(K, generator=g, device=dev)

    def run(x):
        n = x.shape[0]
        o = dict(h=torch.empty_like(x), y=torch.empty_like(x), rstd=torch.empty(n, device=dev), row_amax=torch.empty(n, device=dev),
                 q=torch.full((n, K // 2), 238, dtype=torch.uint8, device=dev), s=torch.full((n, 3), 238, dtype=torch.uint8, device=dev))
        p.nvfp4_rmsnorm(x, w, 1e-5, residual=x, **o)
        return o
    whole = run(x)
    for lo, hi in ((0, 1000), ((1 << 20) - 3, M)):
        for k, v in run(x[lo:hi].clone()).items():
            assert torch.equal(whole[k][lo:hi], v), (k, lo)
    want = 2 * x.double() * ((2 * x.double()).square().mean(1, keepdim=True) + 1e-5) ** -0.5 * w.double()
    assert bool(((whole["y"].double() - want).abs() <= (depth(K) / 2 + 14) * U * want.abs()).all())


# -------------------------------------------------- activation's gradient, sizes
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N", ACT)
def test_bias_gradient_is_the_sum_of_its_rows(M, N, act, dtype):
    """Against FP32 calls of one row each way: the sum over runs of rows, in any order within the bound of a sum."""
    dev = _dev()
    g = torch.Generator(device=dev).manual_seed(M)
    NB = 2 * N if act == "swiglu" else N
    dy, z = torch.randn(M, N, generator=g, device=dev).to(dtype), torch.randn(M, NB, generator=g, device=dev).to(dtype)
    code = getattr(p, "NVFP4_ACT_" + act.upper())
    dz, db = torch.empty(M, NB, device=dev), torch.full((NB,), float("nan"), device=dev)
    p.nvfp4_act_backward(dy.float(), z.float(), code, dz)      # dz unrounded
    p.nvfp4_act_backward(dy, z, code, torch.empty_like(z), dbias=db)
    d = dz.double()
    assert bool(((db.double() - d.sum(0)).abs() <= (M + 2) * U * d.abs().sum(0)).all())
