"""Host-side refusals of the 8-bit integer, layer norm and cache entry points:
every call here is rejected before any HIP call (the addresses are never used)."""
import ctypes

import pytest
import torch

import precision_quantization_row_amd as p

F = ctypes.c_void_p(0x1000)
f = ctypes.c_float
E, U = p.NVFP4_ERR_ARG, p.NVFP4_ERR_UNSUPPORTED


def test_int8_quantize():
    lib = p.load_library()

    def g(x=F, dt=0, M=4, K=8, a=F, q=F):
        return lib.nvfp4_int8_quantize(x, dt, M, K, a, q, None, None)
    for kw in (dict(x=None), dict(dt=2), dict(M=0), dict(K=0), dict(M=-1), dict(K=(1 << 40) + 1), dict(a=None), dict(q=None)):
        assert g(**kw) == E, kw
    assert g(K=(1 << 27) + 1) == U


def test_int8_quantize_rowcol():
    lib = p.load_library()

    def g(x=F, dt=0, M=4, K=8, ra=F, ca=F, qr=F, qc=F):
        return lib.nvfp4_int8_quantize_rowcol(x, dt, M, K, ra, ca, qr, qc, None, None)
    for kw in (dict(x=None), dict(dt=2), dict(M=0), dict(K=0), dict(M=(1 << 40) + 1), dict(ra=None), dict(ca=None),
               dict(qr=None), dict(qc=None)):
        assert g(**kw) == E, kw
    for kw in (dict(K=(1 << 27) + 1), dict(M=(1 << 27) + 1)):
        assert g(**kw) == U, kw


def test_int8_gemm():
    lib = p.load_library()

    def g(a=F, am=1, aa=F, b=F, bm=1, ab=F, M=4, N=4, K=32, bias=None, bd=0, act=0, res=None, z=None, y=F, od=0):
        return lib.nvfp4_int8_gemm(a, am, aa, b, bm, ab, M, N, K, bias, bd, act, res, z, y, od, None, None)
    for kw in (dict(a=None), dict(aa=None), dict(b=None), dict(ab=None), dict(y=None), dict(am=3), dict(bm=-1), dict(M=0),
               dict(N=0), dict(K=0), dict(M=-1), dict(M=(1 << 40) + 1), dict(act=-1), dict(act=5), dict(od=2), dict(bias=F, bd=7)):
        assert g(**kw) == E, kw
    # 2^17 products of -128 by -128 are 2^31: past 32 bits
    for kw in (dict(am=p.NVFP4_AMAX_ROWGROUP), dict(bm=p.NVFP4_AMAX_ROWGROUP), dict(K=1 << 17), dict(N=(1 << 26) + 1),
               dict(M=1 << 32), dict(M=1 << 25, N=1 << 25)):
        assert g(**kw) == U, kw


def test_layernorm():
    lib = p.load_library()

    def g(x=F, res=None, dt=0, w=F, b=None, wd=0, eps=1e-5, M=4, K=8, h=None, y=F, yd=0, mu=None, r=None, fmt=0, q=None, s=None,
          am=None, bound=448.0):
        return lib.nvfp4_layernorm(x, res, dt, w, b, wd, f(eps), M, K, h, y, yd, mu, r, fmt, q, s, am, f(bound), None, None)
    for kw in (dict(x=None), dict(w=None), dict(dt=2), dict(wd=2), dict(yd=2), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(M=0), dict(K=0), dict(y=None), dict(fmt=4, q=F, am=F), dict(fmt=-1), dict(fmt=1),
               dict(q=F, am=F), dict(fmt=1, q=F), dict(fmt=1, q=F, s=F, am=F), dict(fmt=3, q=F, s=F, am=F), dict(fmt=3, q=F),
               dict(fmt=2, q=F, am=F), dict(fmt=2, s=F, am=F), dict(fmt=2, q=F, s=F, am=F, bound=0.0)):
        assert g(**kw) == E, kw
    assert g(K=(1 << 27) + 1) == U


def test_layernorm_backward():
    lib = p.load_library()

    def g(dy=F, h=F, dt=0, w=F, wd=0, mu=F, r=F, dres=None, M=4, K=8, dx=F, dw=None, db=None, ws=None, wb=0):
        return lib.nvfp4_layernorm_backward(dy, h, dt, w, wd, mu, r, dres, M, K, dx, dw, db, ws, wb, None, None)
    need = lib.nvfp4_layernorm_backward_workspace(4, 8)
    assert need >= 2 * 4 * 8
    assert lib.nvfp4_layernorm_backward_workspace(0, 8) == 0
    for kw in (dict(dy=None), dict(h=None), dict(w=None), dict(mu=None), dict(r=None), dict(dx=None), dict(dt=3), dict(wd=3),
               dict(M=0), dict(K=0), dict(dw=F), dict(db=F), dict(dw=F, ws=F, wb=need - 4), dict(db=F, ws=F, wb=need - 4),
               dict(dw=F, db=F, ws=ctypes.c_void_p(0x1008), wb=need)):
        assert g(**kw) == E, kw
    assert g(K=(1 << 27) + 1) == U


CACHE = dict(k=F, ks=1024, v=F, vs=1024, dt=0, T=4, H=8, D=128, fmt=1, bound=448.0, pages=4, size=16, kq=F, ksc=None, ka=F,
             vq=F, vsc=None, va=F, table=F, B=2, cols=2, starts=F, first=None)
BAD = (dict(k=None), dict(v=None), dict(vq=None), dict(va=None), dict(dt=2), dict(T=0), dict(H=0), dict(D=0), dict(B=0),
       dict(cols=0), dict(pages=0), dict(size=0), dict(T=-1), dict(size=(1 << 40) + 1), dict(ks=(1 << 40) + 1), dict(fmt=0), dict(fmt=4),
       dict(kq=None), dict(ka=None), dict(table=None), dict(starts=None), dict(ksc=F), dict(vsc=F), dict(fmt=2),
       dict(fmt=2, ksc=F), dict(fmt=2, ksc=F, vsc=F, bound=0.0), dict(fmt=2, ksc=F, vsc=F, bound=float("nan")))
LIMITS = (dict(D=1025), dict(H=65536), dict(T=1 << 31), dict(B=(1 << 31) - 1))


def test_cache_write():
    lib = p.load_library()

    def g(**kw):
        c = dict(CACHE, **kw)
        return lib.nvfp4_cache_write(c["k"], c["ks"], c["v"], c["vs"], c["dt"], c["T"], c["H"], c["D"], c["fmt"], f(c["bound"]),
                                     c["pages"], c["size"], c["kq"], c["ksc"], c["ka"], c["vq"], c["vsc"], c["va"], c["table"],
                                     c["B"], c["cols"], c["starts"], c["first"], None, None)
    for kw in BAD + (dict(ks=-1), dict(vs=-1)):
        assert g(**kw) == E, kw
    for kw in LIMITS:
        assert g(**kw) == U, kw


def test_cache_read():
    lib = p.load_library()

    def g(**kw):
        c = dict(CACHE, **kw)
        return lib.nvfp4_cache_read(c["kq"], c["ksc"], c["ka"], c["vq"], c["vsc"], c["va"], c["fmt"], f(c["bound"]), c["pages"],
                                    c["size"], c["table"], c["B"], c["cols"], c["starts"], c["first"], c["T"], c["H"], c["D"],
                                    c["k"], c["ks"], c["v"], c["vs"], c["dt"], None, None)
    for kw in BAD + (dict(ks=1023), dict(vs=1023), dict(ks=-1024)):   # rows that would overlap
        assert g(**kw) == E, kw
    for kw in LIMITS:
        assert g(**kw) == U, kw


def test_the_binding_refuses_host_tensors():
    x, a, q = torch.zeros(4, 8), torch.zeros(4), torch.zeros(4, 8, dtype=torch.int8)
    k, t = torch.zeros(2, 1, 8), torch.zeros(1, 1, dtype=torch.int32)
    for call in (lambda: p.nvfp4_int8_quantize(x, a, q), lambda: p.nvfp4_int8_quantize_rowcol(x, a, torch.zeros(8), q, q),
                 lambda: p.nvfp4_int8_gemm(q, 1, a, q, 1, a, 4, 4, 8, torch.zeros(4, 4)),
                 lambda: p.nvfp4_layernorm(x, torch.zeros(8), 1e-5, y=x),
                 lambda: p.nvfp4_layernorm_backward(x, x, torch.zeros(8), a, a, x),
                 lambda: p.nvfp4_cache_write(k, None, q, None, torch.zeros(1, 4, 1), None, None, None, t, t),
                 lambda: p.nvfp4_cache_read(k, None, q, None, torch.zeros(1, 4, 1), None, None, None, t, t)):
        with pytest.raises(ValueError):
            call()
