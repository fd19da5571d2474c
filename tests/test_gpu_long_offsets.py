"""Operands and outputs whose elements lie beyond 32-bit offsets: what the calls
write past the first 2^32 elements or bytes is what calls on those lines alone
give, and sums over them are exact."""
import pytest
import torch

import precision_quantization_row_amd as p
from parity_utils import say

pytestmark = pytest.mark.gpu
BOUND = 512.0 / 6.0   # 1 / (bound 6) is 2^-9


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    p.load_library()
    return torch.device("cuda:0")


def few_codes(g, R, K, fmt, dev):
    """Lines of zeros but for 64 elements each, the last among them; (codes, scales, positions, values)."""
    at = torch.randint(0, K // 2, (R, 64), generator=g, device=dev) * 2 + 1
    at[:, 0] = K - 1
    v = torch.zeros(R, 64, device=dev, dtype=torch.float64)
    v[:] = torch.randint(1, 4, (R, 1), generator=g, device=dev).double()     # one value a line: positions may repeat
    if fmt == "e4m3":
        q = torch.zeros(R, K, dtype=torch.uint8, device=dev)
        q.scatter_(1, at, v.float().to(torch.float8_e4m3fn).view(torch.uint8))
        return q.view(torch.float8_e4m3fn), None, at, v
    q = torch.zeros(R, K // 2, dtype=torch.uint8, device=dev)
    code = (2.0 * v).clamp(max=4).to(torch.uint8) + (v > 2).to(torch.uint8)   # 1 -> 2, 2 -> 4, 3 -> 5
    q.scatter_(1, at // 2, code << 4)
    return q, torch.full((R, K // 16), 0x38, dtype=torch.uint8, device=dev), at, v   # block scales of one


@pytest.mark.parametrize("fmt,M,N", [("e4m3", 1040, 20), ("nvfp4", 2100, 20), ("nvfp4", 20, 2100), ("e4m3", 1040, 1040)])
def test_long_lines(fmt, M, N, dev):
    K = 1 << 22
    say(f"[gpu] long lines {M}x{N}x{K} {fmt}")
    g = torch.Generator(device=dev).manual_seed(1)
    a, sa, pa, va = few_codes(g, M, K, fmt, dev)
    b, sb, pb, vb = few_codes(g, N, K, "nvfp4", dev)
    assert max(a.numel() * a.element_size(), b.numel()) > 1 << 32
    aa, ab = torch.full((M,), 448.0 if fmt == "e4m3" else 512.0, device=dev), torch.full((N,), 512.0, device=dev)
    y = torch.full((M, N), float("nan"), device=dev)
    p.nvfp4_gemm(a, sa, 1, aa, BOUND, b, sb, 1, ab, BOUND, M, N, K, y)
    # each line of the shorter operand, spread out, at the other's positions
    want = torch.zeros(M, N, device=dev, dtype=torch.float64)
    many, few = ((pa, va), (pb, vb)) if M >= N else ((pb, vb), (pa, va))
    line, seen = torch.zeros(K, device=dev, dtype=torch.float64), torch.sort(many[0], 1)
    first = torch.ones_like(seen[0], dtype=torch.bool)
    first[:, 1:] = seen[0][:, 1:] != seen[0][:, :-1]
    for i in range(few[0].shape[0]):
        line.zero_()
        line[few[0][i]] = few[1][i]
        s = (line[seen[0]] * first).sum(1) * many[1][:, 0]
        if M >= N:
            want[:, i] = s
        else:
            want[i] = s
    # (RN(1 / 448) 448 is within 2^-24 of one)
    assert bool(((y.double() - want).abs() <= 3 * 2.0 ** -24 * want).all()) and bool((want > 0).all())


@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_product_of_many_outputs(act, dev):
    M, N, K = 66000, 66000, 32
    say(f"[gpu] many outputs {act}")
    gated = act == "swiglu"
    g = torch.Generator(device=dev).manual_seed(2)
    NB = 2 * N if gated else N
    mk = lambda R: (torch.randint(0, 256, (R, K // 2), generator=g, device=dev).to(torch.uint8),
                    torch.full((R, K // 16), 0x38, dtype=torch.uint8, device=dev), torch.ones(R, device=dev))
    (a, sa, aa), (b, sb, ab) = mk(M), mk(NB)
    code = getattr(p, "NVFP4_ACT_" + act.upper())

    def run(lo, hi):
        m = hi - lo
        y = torch.empty(m, N, dtype=torch.bfloat16, device=dev)
        z = torch.empty(m, NB, dtype=torch.bfloat16, device=dev)
        p.nvfp4_gemm(a[lo:hi], sa[lo:hi], 1, aa[lo:hi], BOUND, b, sb, 1, ab, BOUND, m, N, K, y, z=z, act=code)
        return y, z
    y, z = run(0, M)
    assert y.numel() > 1 << 32
    for lo, hi in ((0, 600), (32768, 33000), (M - 2000, M)):
        yy, zz = run(lo, hi)   # (exact sums: the same bits whichever kernel runs)
        assert torch.equal(y[lo:hi], yy) and torch.equal(z[lo:hi], zz)


def test_norm_and_gradients(dev):
    M, K = 132000, 32768
    say("[gpu] norm and gradients past 2^32 elements")
    g = torch.Generator(device=dev).manual_seed(3)
    x = torch.empty(M, K, dtype=torch.bfloat16, device=dev).normal_(generator=g)
    assert x.numel() > 1 << 32
    w = torch.randn(K, generator=g, device=dev)
    spans = ((0, 300), (65530, 65800), (M - 400, M))

    def norm(x):
        n = x.shape[0]
        o = (torch.empty_like(x), torch.empty(n, K, dtype=torch.float8_e4m3fn, device=dev), torch.empty(n, device=dev),
             torch.empty(n, device=dev))
        p.nvfp4_rmsnorm(x, w, 1e-5, residual=x, h=o[0], q=o[1], row_amax=o[2], rstd=o[3])
        return o
    whole = norm(x)
    for lo, hi in spans:
        assert all(torch.equal(a[lo:hi].view(torch.uint8), b.view(torch.uint8)) for a, b in zip(whole, norm(x[lo:hi])))
    h, rstd = whole[0], whole[3]
    dx, dw = torch.empty_like(x), torch.empty(K, device=dev)
    p.nvfp4_rmsnorm_backward(x, h, w, rstd, dx, dweight=dw)
    want = torch.zeros(K, device=dev, dtype=torch.float64)
    size = torch.zeros_like(want)
    for lo in range(0, M, 4000):
        s = slice(lo, lo + 4000)
        t = x[s].double() * h[s].double() * rstd[s].double()[:, None]
        want += t.sum(0)
        size += t.abs().sum(0)
    assert bool(((dw.double() - want).abs() <= (M / 256 + 40) * 2.0 ** -24 * size).all())
    for lo, hi in spans:
        part = torch.empty_like(x[lo:hi])
        p.nvfp4_rmsnorm_backward(x[lo:hi], h[lo:hi], w, rstd[lo:hi], part)
        assert torch.equal(dx[lo:hi], part)
    del dx, whole
    N = K // 2
    dy = h.view(M, 2, N)[:, 0].contiguous()
    dz, db = torch.empty_like(x), torch.empty(K, device=dev)
    p.nvfp4_act_backward(dy, x, p.NVFP4_ACT_SWIGLU, dz, dbias=db)
    for lo, hi in spans:
        part = torch.empty_like(x[lo:hi])
        p.nvfp4_act_backward(dy[lo:hi], x[lo:hi], p.NVFP4_ACT_SWIGLU, part)
        assert torch.equal(dz[lo:hi], part)
    # of the FP32 values, each within half a BF16 step of the stored one
    total, size = torch.zeros(K, device=dev, dtype=torch.float64), torch.zeros(K, device=dev, dtype=torch.float64)
    for lo in range(0, M, 4000):
        d = dz[lo:lo + 4000].double()
        total += d.sum(0)
        size += d.abs().sum(0)
    assert bool(((db.double() - total).abs() <= (2.0 ** -8 + (M / 4 + 40) * 2.0 ** -24) * 1.01 * size).all())
