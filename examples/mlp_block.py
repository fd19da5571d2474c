"""A gated MLP block in row-scaled NVFP4: one training step and one decode step.

  h = x + r;  y = rmsnorm(h) * w;  a = silu(y Wg^T) * (y Wu^T);  out = a Wd^T + h

Training quantizes each matrix once in both directions (nvfp4_quantize_rowcol);
the rowwise copies feed the forward products, the columnwise copies the
gradients'. Decoding norms a few tokens straight into 8-bit lines. Every
product is checked against its dequantized operands.

  python examples/mlp_block.py [tokens] [width] [hidden]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import precision_quantization_row_amd as p  # noqa: E402

BOUND, EPS, LINE = 448.0, 1e-5, p.NVFP4_AMAX_LINE


class Packed:
    """Both NVFP4 copies of a matrix: row (lines = rows) and col (lines = columns)."""

    def __init__(self, x):
        M, K = x.shape
        o = p.empty_outputs(M, K, x.device)
        ra, ca = torch.empty(M, device=x.device), torch.empty(K, device=x.device)
        p.nvfp4_quantize_rowcol(x, ra, ca, BOUND, o["q_row"], o["s_row"], o["q_col"], o["s_col"])
        self.row = (o["q_row"], o["s_row"], ra, K)
        self.col = (o["q_col"], o["s_col"], ca, M)


def dequantized(lines):
    q, s, amax, length = lines
    if s is None:
        return q.float() * (amax / 448.0)[:, None]
    y = torch.empty(amax.numel(), length, device=q.device)
    p.nvfp4_dequantize(q, s, amax.numel(), length, LINE, amax, BOUND, y)
    return y


worst = {}


def product(name, A, B, out_dtype=torch.bfloat16, **kw):
    """act(A B^T) + residual of two sets of lines along the same axis."""
    (a, sa, aa, K), (b, sb, ab, _) = A, B
    gated = kw.get("act") == p.NVFP4_ACT_SWIGLU
    M, N = aa.numel(), ab.numel() // (2 if gated else 1)
    y = torch.empty(M, N, dtype=out_dtype, device=a.device)
    p.nvfp4_gemm(a, sa, LINE, aa, BOUND, b, sb, LINE, ab, BOUND, M, N, K, y, **kw)
    want = dequantized(A) @ dequantized(B).t()
    if gated:
        want = torch.nn.functional.silu(want[:, :N]) * want[:, N:]
    if kw.get("residual") is not None:
        want = want + kw["residual"].float()
    worst[name] = float((y.float() - want).norm() / want.norm())
    return y


def train_step(x, r, dout, w, W1, W2):
    """Forward and backward; returns (out, dx, dw, dW1, dW2). x's gradient is r's too."""
    T, D = x.shape
    h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device=x.device)
    p.nvfp4_rmsnorm(x, w, EPS, residual=r, h=h, y=y, rstd=rstd)
    py, pw1, pw2 = Packed(y), Packed(W1), Packed(W2)
    z = torch.empty(T, W1.shape[0], dtype=x.dtype, device=x.device)
    a = product("gate and up", py.row, pw1.row, act=p.NVFP4_ACT_SWIGLU, z=z)
    pa = Packed(a)
    out = product("down", pa.row, pw2.row, residual=h)

    pd = Packed(dout)
    da = product("down, data gradient", pd.row, pw2.col)
    dW2 = product("down, weight gradient", pd.col, pa.col, torch.float32)
    dz = torch.empty_like(z)
    p.nvfp4_act_backward(da, z, p.NVFP4_ACT_SWIGLU, dz)
    pz = Packed(dz)
    dy = product("gate and up, data gradient", pz.row, pw1.col)
    dW1 = product("gate and up, weight gradient", pz.col, py.col, torch.float32)
    dx, dw = torch.empty_like(x), torch.empty(D, device=x.device)
    p.nvfp4_rmsnorm_backward(dy, h, w, rstd, dx, dweight=dw, dres=dout)
    return out, dx, dw, dW1, dW2


def decode_step(x, r, w, pw1, pw2):
    """A few tokens: the norm writes 8-bit lines, the activations go on in NVFP4."""
    T, D = x.shape
    h, amax = torch.empty_like(x), torch.empty(T, device=x.device)
    q = torch.empty(T, D, dtype=torch.float8_e4m3fn, device=x.device)
    p.nvfp4_rmsnorm(x, w, EPS, residual=r, h=h, q=q, row_amax=amax)
    a = product("decode, gate and up", (q, None, amax, D), pw1.row, act=p.NVFP4_ACT_SWIGLU)
    return product("decode, down", Packed(a).row, pw2.row, residual=h)


def main(tokens=1024, width=1024, hidden=2816, device="cuda"):
    g = torch.Generator().manual_seed(0)
    rand = lambda *s, k=1.0: (torch.randn(*s, generator=g) * k).to(device).bfloat16()
    x, r, dout = rand(tokens, width), rand(tokens, width), rand(tokens, width)
    w = (1 + 0.1 * torch.randn(width, generator=g)).to(device).bfloat16()
    W1, W2 = rand(2 * hidden, width, k=width ** -0.5), rand(width, hidden, k=hidden ** -0.5)
    out, *_ = train_step(x, r, dout, w, W1, W2)
    few = decode_step(x[:4].clone(), r[:4].clone(), w, Packed(W1), Packed(W2))
    # the 8-bit tokens differ from the NVFP4 ones by the quantization alone
    worst["decode against training"] = float((few.float() - out[:4].float()).norm() / out[:4].float().norm())
    torch.cuda.synchronize()
    return dict(worst)


if __name__ == "__main__":
    for name, err in main(*map(int, sys.argv[1:4])).items():
        print(f"{name:32s} relative error {err:.2e}")
