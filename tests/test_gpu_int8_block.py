"""The operators together, as an attention layer's front and a training step use
them: the layer norm into 8-bit tokens, the fused projection, its keys and
values into the cache and back; and the three products of training with the
norm's gradient."""
import pytest
import torch

import precision_quantization_row_amd as p
from product_utils import DEV

pytestmark = pytest.mark.gpu
LINE, BF, EPS = p.NVFP4_AMAX_LINE, torch.bfloat16, 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    p.load_library()


def both(x):
    R, C = x.shape
    o = (torch.empty(R, C, dtype=torch.int8, device=DEV), torch.empty(R, device=DEV),
         torch.empty(C, R, dtype=torch.int8, device=DEV), torch.empty(C, device=DEV))
    p.nvfp4_int8_quantize_rowcol(x, o[1], o[3], o[0], o[2])
    return (o[0], o[1]), (o[2], o[3])


def product(A, B, dtype=BF, **kw):
    (a, aa), (b, ab) = A, B
    y = torch.empty(a.shape[0], b.shape[0], dtype=dtype, device=DEV)
    p.nvfp4_int8_gemm(a, LINE, aa, b, LINE, ab, a.shape[0], b.shape[0], a.shape[1], y, **kw)
    return y


def values(lines):
    return lines[0].double() * (lines[1].double() / 127)[:, None]


@pytest.mark.parametrize("fmt", [torch.int8, torch.float8_e4m3fn, torch.uint8])
def test_prompt_then_decode(fmt):
    """A prompt of two sequences, then single tokens; what is read back is what was projected, but for the cache's codes."""
    g = torch.Generator(device=DEV).manual_seed(0)
    W, H, D, size = 512, 4, 64, 16
    heads = 8                                    # of queries
    N = (heads + 2 * H) * D
    w_n, b_n = 1 + 0.1 * torch.randn(W, generator=g, device=DEV), 0.1 * torch.randn(W, generator=g, device=DEV)
    wq, wa = torch.empty(N, W, dtype=torch.int8, device=DEV), torch.empty(N, device=DEV)
    weight = torch.randn(N, W, generator=g, device=DEV) * W ** -0.5
    p.nvfp4_int8_quantize(weight, wa, wq)
    pages = 24
    width = D // 2 if fmt == torch.uint8 else D
    mk = lambda: (torch.zeros(pages, size, H, width, dtype=torch.uint8, device=DEV).view(fmt),
                  torch.zeros(pages, size, H, D // 16, dtype=torch.uint8, device=DEV) if fmt == torch.uint8 else None,
                  torch.zeros(pages, size, H, device=DEV))
    kc, vc = mk(), mk()
    table = torch.randperm(pages, generator=g, device=DEV).int().view(2, -1)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)
    seen = [[], []]
    done = [0, 0]
    for lengths in ((37, 50), (1, 1), (1, 1), (0, 1)):
        T = sum(lengths)
        x, r = torch.randn(T, W, generator=g, device=DEV).to(BF), torch.randn(T, W, generator=g, device=DEV).to(BF)
        h, q, a = torch.empty_like(x), torch.empty(T, W, dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
        p.nvfp4_layernorm(x, w_n, EPS, bias=b_n, residual=r, h=h, q=q, row_amax=a)
        qkv = product((q, a), (wq, wa))
        # the layer in 64 bits: norm, projection of the dequantized weights; apart by the tokens' codes (half a step of
        # amax / 127 an element, W of them of random sign) and BF16's rounding
        h64 = x.double() + r.double()
        d = h64 - h64.mean(1, keepdim=True)
        y64 = d * (d.square().mean(1, keepdim=True) + EPS) ** -0.5 * w_n.double() + b_n.double()
        want = y64 @ values((wq, wa)).t()
        assert float((qkv.double() - want).norm() / want.norm()) < 0.5 * float((a.double() / 127).max()) + 2 ** -8
        k, v = (qkv[:, (heads + i * H) * D:(heads + (i + 1) * H) * D].unflatten(1, (H, D)) for i in (0, 1))
        starts = i32(0, lengths[0], T)
        p.nvfp4_cache_write(k, v, *kc, *vc, table, starts, first=i32(*done))
        for b in (0, 1):
            lo, hi = (0, lengths[0]) if b == 0 else (lengths[0], T)
            seen[b].append((k[lo:hi].float(), v[lo:hi].float()))
            done[b] += lengths[b]
        total = sum(done)
        ko, vo = torch.empty(total, H, D, dtype=BF, device=DEV), torch.empty(total, H, D, dtype=BF, device=DEV)
        p.nvfp4_cache_read(ko, vo, *kc, *vc, table, i32(0, done[0], total))
        for i, got in ((0, ko), (1, vo)):
            was = torch.cat([t[i] for b in (0, 1) for t in seen[b]])
            top = was.abs().amax(2, keepdim=True)
            # half a step: int8 a / 254; E4M3 2^-4 of the value, or half its least step, a / 448 2^-10; E2M1 up to
            # 1 of the block's 6, whose scale is off by 2^-4 (and saturates there); BF16 and a few FP32 roundings besides
            step = {torch.int8: top / 254, torch.float8_e4m3fn: was.abs() * 2 ** -4 + top / 448 * 2 ** -10,
                    torch.uint8: top / 6 * (1 + 2 ** -3) + top * 2 ** -3}[fmt]
            assert bool(((got.float() - was).abs() <= step * 1.001 + 2 ** -8 * 1.1 * (was.abs() + step)).all())


def test_training_step():
    """out = (norm(x + r) W^T + c) and its gradients through the three products: against the same formulas in 64 bits of the
    dequantized operands."""
    g = torch.Generator(device=DEV).manual_seed(1)
    T, W, N = 300, 256, 384
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)
    x, r, dout = rand(T, W).to(BF), rand(T, W).to(BF), rand(T, N).to(BF)
    w, b, weight, c = (1 + 0.1 * rand(W)).to(BF), rand(W).to(BF), (rand(N, W) * W ** -0.5).to(BF), rand(N)
    h, y = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    p.nvfp4_layernorm(x, w, EPS, bias=b, residual=r, h=h, y=y, mean=mean, rstd=rstd)
    (yr, yc), (wr, wc), (dr, dc) = both(y), both(weight), both(dout)
    out, dy, dW = product(yr, wr, bias=c), product(dr, wc), product(dc, yc, torch.float32)
    dx, dw, db = torch.empty_like(x), torch.empty(W, device=DEV), torch.empty(W, device=DEV)
    p.nvfp4_layernorm_backward(dy, h, w, mean, rstd, dx, dweight=dw, dbias=db, dres=x)
    close = lambda got, want, tol: float((got.double() - want).norm() / want.norm()) < tol
    assert close(out, values(yr) @ values(wr).t() + c.double(), 2 ** -8)
    assert close(dy, values(dr) @ values(wc).t(), 2 ** -8) and close(dW, values(dc) @ values(yc).t(), 1e-6)
    # the norm's gradient of that dy, in 64 bits, from autograd's formulas
    leaf = [t.double().requires_grad_() for t in (h, w, b)]
    d = leaf[0] - leaf[0].mean(1, keepdim=True)
    (d * (d.square().mean(1, keepdim=True) + EPS) ** -0.5 * leaf[1] + leaf[2]).backward(dy.double())
    # (the kernel's mean and rstd are of the FP32 sum, h is its rounding to BF16: 2^-8 an element)
    assert close(dx, leaf[0].grad + x.double(), 2 ** -6) and close(dw, leaf[1].grad, 2 ** -6) and close(db, leaf[2].grad, 1e-6)
    # and the products' straight-through gradients are those of the unquantized formulas, but for the codes: 1 / 254 of
    # each line's amax, some 4 deviations, an element
    assert close(dW, dout.double().t() @ y.double(), 0.05) and close(dy, dout.double() @ weight.double(), 0.05)
