"""The norm and its gradient at ordinary hidden sizes: every form of the row passes (rows of up to 2,048, 4,096
and 8,192 columns in registers, wider ones beyond), with fewer rows than workgroups and with several rows to
each."""
import pytest
import torch

import blockwise_fp8_gemm_amd as pf
from fused_ref import U, bf16, check_blocks, check_dual, close_bf16, f64, norm, norm_bwd

pytestmark = pytest.mark.gpu

EPS = 1e-6
WIDTHS = [1024, 2040, 2056, 2560, 4096, 4100, 5120, 6144, 8192, 8200]
# more rows than the forward's 4,096 or 2,048 workgroups and the gradient's 512 to 1,024
MANY = [(4200, 512), (2100, 2560), (2100, 4100)]
MANY_BWD = [(5000, 256), (3000, 1024), (2100, 2048), (1100, 2560), (1100, 4100), (1030, 8200)]


def shares(tokens, cols):
    """Workgroups of the gradient's row pass, each of which adds up one share of dw."""
    most = 512
    if cols <= 2048 and tokens > 4 * most:
        most = min((tokens + 3) // 4, 1024)
    return min((tokens + 1) // 2, most)


def dw_tolerance(dy, z, r):
    """dw's terms dy (z r): z r is rounded, then a term passes its share's rows one after the other (products
    are not rounded, they are fused), the shares that one of 16 threads adds, and four additions of those."""
    tokens, cols = z.shape
    g = shares(tokens, cols)
    steps = 1 + -(-tokens // g) + -(-g // 16) + 4
    return (dy * z * r[:, None]).abs().sum(0) * (steps + 1) * U + 2.0 ** -147


def weight(cols, seed, dtype, dev):
    gen = torch.Generator().manual_seed(seed)
    return (1.0 + 0.2 * torch.randn((cols,), generator=gen)).to(dtype).to(dev)


def stream(tokens, cols, seed, dev):
    r = bf16(tokens, cols, 2.0, seed, dev, 16)
    r[:, cols // 2] *= 100
    r[0] = 0
    return r


@pytest.mark.parametrize("tokens,cols", [(1, w) for w in WIDTHS] + [(130, w) for w in WIDTHS] + MANY)
def test_forward(dev, tokens, cols):
    x, res = bf16(tokens, cols, 1.0, 1, dev, 16), stream(tokens, cols, 2, dev)
    x[0] = 1.0          # no zero row here: the stream's is zero alone
    w = weight(cols, 3, torch.bfloat16 if cols % 3 else torch.float32, dev)
    z, r, h, q, s = pf.puro_fp8_rmsnorm_quant_act(x, w, res, eps=EPS, store_h=True)
    dual = pf.puro_fp8_rmsnorm_quant_dual(x, w, res, eps=EPS, store_h=True)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((z, r, h, q, s), dual[:5]))
    Z = f64((x.float() + res.float()).bfloat16())
    assert torch.equal(f64(z), Z)
    n, tol, want, rel = norm(Z, f64(w), EPS)
    assert bool(((f64(r) - want).abs() <= rel * want).all())
    check_dual(n, tol, *dual[3:], "norm")
    close_bf16(h, n, tol, "h")
    # without a residual
    z, r, _, q, s = pf.puro_fp8_rmsnorm_quant_act(res, w, eps=EPS)
    torch.cuda.synchronize()
    n, tol, want, rel = norm(f64(res), f64(w), EPS)
    assert z.data_ptr() == res.data_ptr() and bool(((f64(r) - want).abs() <= rel * want).all())
    check_blocks(n, tol, q, s, "norm of x")


@pytest.mark.parametrize("tokens,cols", [(1, w) for w in WIDTHS] + [(130, w) for w in WIDTHS] + MANY_BWD)
def test_gradient(dev, tokens, cols):
    z, dy = stream(tokens, cols, 4, dev), bf16(tokens, cols, 1e-3, 5, dev)
    dres = bf16(tokens, cols, 1e-3, 6, dev, 48) if cols % 4 == 0 else None
    w = weight(cols, 7, torch.float32 if cols % 3 else torch.bfloat16, dev)
    r = torch.rsqrt(z.double().square().mean(1) + EPS).float()
    dx, dw, qr, sr, qt, st = pf.puro_fp8_rmsnorm_bwd_quant_dual(dy, z, r, w, dres)
    torch.cuda.synchronize()
    Y, Z, R = f64(dy), f64(z), f64(r)
    ex, tol, ew, _ = norm_bwd(Y, Z, R, f64(w), f64(dres) if dres is not None else None)
    close_bf16(dx, ex, tol, "dx")
    assert bool(((f64(dw) - ew).abs() <= dw_tolerance(Y, Z, R)).all())
    check_dual(ex, tol, qr, sr, qt, st, "dx")
    again = pf.puro_fp8_rmsnorm_bwd_quant_dual(dy, z, r, w, dres)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, qr, sr, qt, st), again))


def test_shares_are_the_workspaces(dev):
    """The workspace holds a number a token and the shares, rows padded to 16: what dw_tolerance assumes of them."""
    for tokens, cols in [(1, 1), (130, 2056)] + MANY_BWD:
        want = -(-tokens * 4 // 256) * 256 + shares(tokens, cols) * (-(-cols // 16) * 16) * 4
        assert pf.puro_fp8_rmsnorm_bwd_workspace_size(tokens, cols) == want
