"""The norm's gradient where the products of its inputs leave FP32 although the formula's own values do not:
xh = z r is of order one whatever z's size, so w dy xh is the size of dy and r the inverse of z's."""
import pytest
import torch

import blockwise_fp8_gemm_amd as pf
from fused_ref import bf16, check_dual, close_bf16, f64, norm_bwd

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
