"""Host-side refusals of the product, norm and gradient entry points: every
call here is rejected before any HIP call (the addresses are never used)."""
import ctypes

import precision_quantization_row_amd as p

F = ctypes.c_void_p(0x1000)
f = ctypes.c_float
E, U = p.NVFP4_ERR_ARG, p.NVFP4_ERR_UNSUPPORTED


def test_gemm():
    lib = p.load_library()

    def g(fmt=2, a=F, sa=F, am=1, aa=F, abound=448.0, b=F, sb=F, bm=1, ab=F, bbound=448.0, M=4, N=4, K=32,
          bias=None, bd=0, act=0, res=None, z=None, y=F, od=0):
        return lib.nvfp4_gemm(fmt, a, sa, am, aa, f(abound), b, sb, bm, ab, f(bbound), M, N, K, bias, bd, act, res, z,
                              y, od, None, None)
    for kw in (dict(a=None), dict(sa=None), dict(aa=None), dict(b=None), dict(sb=None), dict(ab=None), dict(y=None),
               dict(fmt=0), dict(fmt=3), dict(fmt=1), dict(am=3), dict(bm=-1), dict(abound=0.0), dict(abound=449.0),
               dict(bbound=float("nan")), dict(bbound=-1.0), dict(M=0), dict(N=0), dict(K=0), dict(M=-1),
               dict(M=(1 << 40) + 1), dict(act=-1), dict(act=5), dict(od=2), dict(bias=F, bd=7)):
        assert g(**kw) == E, kw
    for kw in (dict(am=p.NVFP4_AMAX_ROWGROUP), dict(bm=p.NVFP4_AMAX_ROWGROUP), dict(K=(1 << 23) + 1),
               dict(N=(1 << 26) + 1), dict(M=1 << 32), dict(M=1 << 25, N=1 << 25)):
        assert g(**kw) == U, kw


def test_act_backward():
    lib = p.load_library()

    def g(dy=F, z=F, dt=0, M=4, N=8, act=1, dz=F, db=None, ws=None, wb=0):
        return lib.nvfp4_act_backward(dy, z, dt, M, N, act, dz, db, ws, wb, None, None)
    need = lib.nvfp4_act_backward_workspace(4, 8, 1)
    assert need == 4 * 8 and lib.nvfp4_act_backward_workspace(4, 8, 4) == 2 * need
    for kw in (dict(dy=None), dict(z=None), dict(dz=None), dict(dt=2), dict(M=0), dict(N=0), dict(act=5), dict(act=-1),
               dict(db=F), dict(db=F, ws=F, wb=need - 1), dict(db=F, ws=ctypes.c_void_p(0x1004), wb=need)):
        assert g(**kw) == E, kw
    assert g(N=(1 << 27) + 1) == U


def test_rmsnorm():
    lib = p.load_library()

    def g(x=F, res=None, dt=0, w=F, wd=0, eps=1e-5, M=4, K=8, h=None, y=F, yd=0, r=None, fmt=0, q=None, s=None, am=None,
          bound=448.0):
        return lib.nvfp4_rmsnorm(x, res, dt, w, wd, f(eps), M, K, h, y, yd, r, fmt, q, s, am, f(bound), None, None)
    for kw in (dict(x=None), dict(w=None), dict(dt=2), dict(wd=2), dict(yd=2), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(M=0), dict(K=0), dict(y=None), dict(fmt=3, q=F, am=F), dict(fmt=1), dict(q=F, am=F),
               dict(fmt=1, q=F), dict(fmt=1, q=F, s=F, am=F), dict(fmt=2, q=F, am=F), dict(fmt=2, s=F, am=F),
               dict(fmt=2, q=F, s=F, am=F, bound=0.0)):
        assert g(**kw) == E, kw
    assert g(K=(1 << 27) + 1) == U


def test_rmsnorm_backward():
    lib = p.load_library()

    def g(dy=F, h=F, dt=0, w=F, wd=0, r=F, dres=None, M=4, K=8, dx=F, dw=None, ws=None, wb=0):
        return lib.nvfp4_rmsnorm_backward(dy, h, dt, w, wd, r, dres, M, K, dx, dw, ws, wb, None, None)
    need = lib.nvfp4_rmsnorm_backward_workspace(4, 8)
    assert need == 4 * 4 * 8
    for kw in (dict(dy=None), dict(h=None), dict(w=None), dict(r=None), dict(dx=None), dict(dt=3), dict(wd=3), dict(M=0),
               dict(K=0), dict(dw=F), dict(dw=F, ws=F, wb=need - 4), dict(dw=F, ws=ctypes.c_void_p(0x1008), wb=need)):
        assert g(**kw) == E, kw
    assert g(K=(1 << 27) + 1) == U
