"""The norm with the smallest eps, and its gradient where the products of its inputs leave FP32 although the formula's own values do not:
xh = z r is of order one whatever z's size, so w dy xh is the size of dy and r the inverse of z's."""
import pytest
import torch

import blockwise_fp8_gemm_amd as pf
from fused_ref import U, bf16, check_blocks, check_dual, close_bf16, f64, norm, norm_bwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,cols", [(1, 1), (5, 130), (130, 2048), (9, 4100), (3, 9000)])
@pytest.mark.parametrize("z_pow,dy_pow", [(60, 68), (-60, -84), (-60, 30), (40, -100)])
def test_gradient_of_far_magnitudes(dev, tokens, cols, z_pow, dy_pow):
    """2^60 x 2^68 passes FP32's range, 2^-60 x 2^-84 falls into its subnormals; dx is dy over z's size."""
    z = bf16(tokens, cols, 1.0, 1, dev) * 2.0 ** z_pow
    dy = bf16(tokens, cols, 1.0, 2, dev) * 2.0 ** dy_pow
    z, dy = (pf.empty_2d(tokens, cols, torch.bfloat16, dev).copy_(t) for t in (z, dy))
    gen = torch.Generator().manual_seed(3)
    w = (1 + 0.2 * torch.randn((cols,), generator=gen)).to(dev)
    r = torch.rsqrt(z.double().square().mean(1)).float()
    dx, dw, qr, sr, qt, st = pf.puro_fp8_rmsnorm_bwd_quant_dual(dy, z, r, w)
    torch.cuda.synchronize()
    ex, tol, ew, dtol = norm_bwd(f64(dy), f64(z), f64(r), f64(w), None)
    close_bf16(dx, ex, tol, "dx")
    # one token's shares: no more additions than the old bound counts
    assert bool(((f64(dw) - ew).abs() <= dtol).all())
    check_dual(ex, tol, qr, sr, qt, st, "dx")


@pytest.mark.parametrize("z_pow", [-70, -62, -75])
@pytest.mark.parametrize("cols", [1, 130, 2048, 9000])
def test_smallest_eps(dev, cols, z_pow):
    """eps = 2^-126, the smallest taken, beside squares that are subnormal (2^-140, 2^-124, 2^-150): each is off by
    2^-150 at most, 2^-24 of eps, and so is their mean."""
    eps = 2.0 ** -126
    x = pf.empty_2d(40, cols, torch.bfloat16, dev).copy_(bf16(40, cols, 1.0, 5, dev) * 2.0 ** z_pow)
    w = torch.ones((cols,), device=dev)
    z, r, _, q, s = pf.puro_fp8_rmsnorm_quant_act(x, w, eps=eps)
    torch.cuda.synchronize()
    n, tol, want, rel = norm(f64(x), f64(w), eps)
    assert bool(((f64(r) - want).abs() <= (rel + U) * want).all())
    check_blocks(n, tol + n.abs() * U, q, s, "norm")


def test_subnormal_eps_is_refused(dev):
    x, w = bf16(4, 128, 1.0, 6, dev), torch.ones((128,), device=dev)
    for call in (pf.puro_fp8_rmsnorm_quant_act, pf.puro_fp8_rmsnorm_quant_dual):
        for eps in (2.0 ** -127, 1e-40, 2.0 ** -149):
            with pytest.raises(pf.PuroError, match="out of range"):
                call(x, w, eps=eps)
