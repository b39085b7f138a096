"""The orthogonalisation over FP32's whole range: the factor s / (|G| + eps) that brings X to its scale reaches
from 2^-142 to 2^156, which one FP32 number does not hold."""
import pytest
import torch

import blockwise_fp8_gemm_amd as pf
from test_gpu_newton_schulz import check, gradient

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [1e-37, 2.0 ** -126, 1e-40, 2.0 ** -149])
@pytest.mark.parametrize("rows,cols", [(1, 1), (64, 4096), (300, 130)])
def test_zeros_give_zeros(dev, rows, cols, eps):
    for dtype in (torch.float32, torch.bfloat16):
        z = torch.zeros((rows, (cols + 15) // 16 * 16), dtype=dtype, device=dev)[:, :cols]
        out, = pf.puro_fp8_newton_schulz_grouped([z], eps=eps)
        torch.cuda.synchronize()
        assert not bool(out.isnan().any()) and not bool(out.any())


@pytest.mark.parametrize("rows,cols", [(96, 224), (300, 130), (128, 128)])
@pytest.mark.parametrize("power", [-120, -100, 110, 138])
def test_smallest_and_largest_elements(dev, rows, cols, power):
    """From FP32 subnormals (1e-4 x 2^-120: some 17 bits of the largest) to 1e38.  The factors are powers of two,
    so the large ones' results are those of the gradient itself, bit for bit."""
    g = gradient(rows, cols, 511, torch.float32, dev, "normal")
    big = torch.zeros((rows, (cols + 15) // 16 * 16), device=dev)[:, :cols]
    big.copy_(g * 2.0 ** (power // 2) * 2.0 ** (power - power // 2))
    assert bool(torch.isfinite(big).all())
    out, = pf.puro_fp8_newton_schulz_grouped([big], eps=2.0 ** -149)
    torch.cuda.synchronize()
    check(out, big, eps=2.0 ** -149)
    if power > 0:
        assert torch.equal(out, pf.puro_fp8_newton_schulz_grouped([g], eps=2.0 ** -149)[0])
