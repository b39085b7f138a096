"""The largest extents of the norm and activation-gradient calls, one at a time: 2^23 tokens of a few
columns and a few tokens of 2^23 columns, checked on slices that include the ends; and the largest
matrix of the orthogonalisation, on a product whose result is known."""
import pytest
import torch

import blockwise_fp8_gemm_amd as pf
from fused_ref import check_blocks, f64, norm, norm_bwd, swiglu_bwd

pytestmark = pytest.mark.gpu

EPS = 1e-6
MOST = 1 << 23


def rand(rows, cols, std, seed, dev):
    gen = torch.Generator(device=dev).manual_seed(seed)
    return (torch.randn((rows, cols), generator=gen, device=dev) * std).bfloat16()


@pytest.mark.parametrize("cols", [16, 144])
def test_most_tokens(dev, cols):
    tokens = MOST - (40 if cols == 144 else 0)
    x, dy = rand(tokens, cols, 1.0, 1, dev), rand(tokens, cols, 1.0, 2, dev)
    w = 1 + 0.1 * torch.rand((cols,), device=dev)
    z, r, _, q, s, qt, st = pf.puro_fp8_rmsnorm_quant_dual(x, w, eps=EPS)
    dx, dw, qr, sr, qxt, sxt = pf.puro_fp8_rmsnorm_bwd_quant_dual(dy, z, r, w)
    outs = pf.puro_fp8_swiglu_bwd_quant_dual(dy, x, x)
    torch.cuda.synchronize()
    last = tokens // 128 * 128 - 128
    for lo, hi in ((0, 128), (1 << 22, (1 << 22) + 128), (last, tokens)):
        nt = slice(lo // 128, -(-hi // 128))
        X, D, R = f64(x[lo:hi]), f64(dy[lo:hi]), f64(r[lo:hi])
        n, tol, rs, rel = norm(X, f64(w), EPS)
        assert bool(((R - rs).abs() <= rel * rs).all())
        check_blocks(n, tol, q[lo:hi], s[lo:hi], "norm rows")
        check_blocks(n.t(), tol.t(), qt[:, lo:hi], st[:, nt], "norm tokens")
        ex, tx, _, _ = norm_bwd(D, X, R, f64(w), None)
        check_blocks(ex, tx, qr[lo:hi], sr[lo:hi], "dx rows")
        check_blocks(ex.t(), tx.t(), qxt[:, lo:hi], sxt[:, nt], "dx tokens")
        dg, du, tg, tu = swiglu_bwd(D, X, X)
        for v, t, o in ((dg, tg, outs[0]), (du, tu, outs[1])):
            check_blocks(v, t, o[0][lo:hi], o[1][lo:hi], "activation rows")
            check_blocks(v.t(), t.t(), o[2][:, lo:hi], o[3][:, nt], "activation tokens")
    # dw over all tokens, in 64 bits on the GPU; every share adds tokens / 1024 terms one after the other
    exact, mag = torch.zeros(cols, dtype=torch.float64, device=dev), torch.zeros(cols, dtype=torch.float64, device=dev)
    for lo in range(0, tokens, 1 << 20):
        p = dy[lo:lo + (1 << 20)].double() * x[lo:lo + (1 << 20)].double() * r[lo:lo + (1 << 20), None].double()
        exact += p.sum(0)
        mag += p.abs().sum(0)
    assert bool(((dw.double() - exact).abs() <= mag * (tokens // 1024 + 64 + 8 + 4) * 2.0 ** -24).all())


@pytest.mark.parametrize("cols", [MOST, MOST - 24])
def test_most_columns(dev, cols):
    tokens = 3
    x, res, dy = (torch.zeros((tokens, MOST), dtype=torch.bfloat16, device=dev)[:, :cols] for _ in range(3))
    for k, t in enumerate((x, res, dy)):
        t.copy_(rand(tokens, cols, 1.0, 10 + k, dev))
    w = 1 + 0.1 * torch.rand((cols,), device=dev)
    z, r, _, q, s = pf.puro_fp8_rmsnorm_quant_act(x, w, res, eps=EPS)
    dx, dw, qr, sr, qxt, sxt = pf.puro_fp8_rmsnorm_bwd_quant_dual(dy, z, r, w, res)
    torch.cuda.synchronize()
    Z = f64((x.float() + res.float()).bfloat16())
    assert torch.equal(f64(z), Z)
    n, tol, rs, rel = norm(Z, f64(w), EPS)
    assert bool(((f64(r) - rs).abs() <= rel * rs).all())
    ex, tx, ew, tw = norm_bwd(f64(dy), Z, f64(r), f64(w), f64(res))
    assert bool(((f64(dw) - ew).abs() <= tw).all())
    for lo, hi in ((0, 1024), (8192, 8192 + 1024), (cols // 128 * 128 - 1024, cols)):
        nb = slice(lo // 128, -(-hi // 128))
        check_blocks(n[:, lo:hi], tol[:, lo:hi], q[:, lo:hi], s[:, nb], "norm")
        check_blocks(ex[:, lo:hi], tx[:, lo:hi], qr[:, lo:hi], sr[:, nb], "dx rows")
        check_blocks(ex[:, lo:hi].t(), tx[:, lo:hi].t(), qxt[lo:hi], sxt[lo:hi], "dx tokens")


def test_largest_matrix(dev):
    """A 16384 x 16384 gradient of orthogonal rows times a number: X X^T stays a multiple of the identity, so
    every singular value follows the quintic from 1 / 128 on."""
    n = 16384
    signs = torch.ones((1, 1), device=dev)
    while signs.shape[0] < n:      # Sylvester's construction: rows of +-1, orthogonal
        signs = torch.cat((torch.cat((signs, signs), 1), torch.cat((signs, -signs), 1)), 0)
    out, = pf.puro_fp8_newton_schulz_grouped([signs])
    torch.cuda.synchronize()
    s = 1 / 128                    # |G|_F = n, G's singular values are sqrt(n)
    for _ in range(5):
        s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
    # Relative errors.  d log f / d log s is 1.00, 1.00, 0.98, 0.71, -1.57 at the five steps' values, so one made
    # at a step's end has grown 1.09, 1.09, 1.11, 1.57, 1 times at the last.  A step makes two half steps of FP16
    # at most (X as an operand, B): 2 x 5.9, and 1.1 for the input's.  A's diagonal adds 16384 terms in FP32,
    # 2^-10 of it at most, and (d log f / d log s - 1) / 2 of that reaches the step's value: 1.5 x 2^-10 from
    # the last two.  In all 16 x 2^-11, and the result's own rounding to BF16.
    want = s / 128
    off = (out.float() - want * signs).abs()
    assert float(off.max()) <= want * (16 * 2.0 ** -11 + 2.0 ** -8), (float(off.max()), want)
