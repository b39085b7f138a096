"""GPU parity of the gated activation's gradient against its 64-bit formula (tolerances derived in
fused_ref), separate and joined outputs, both token-copy layouts and scale rules."""
import numpy as np
import pytest
import torch

import blockwise_fp8_gemm_amd as pf
from fused_ref import bf16, check_dual, f64, swiglu_bwd

pytestmark = pytest.mark.gpu

SIZES = [(1, 1), (1, 128), (5, 130), (127, 256), (128, 128), (129, 384), (300, 1000)]


@pytest.mark.parametrize("pow2", [False, True], ids=["amax", "pow2"])
@pytest.mark.parametrize("transpose_out", [True, False], ids=["nt", "tn"])
@pytest.mark.parametrize("tokens,cols", SIZES)
def test_gradient(dev, tokens, cols, transpose_out, pow2):
    gate, up = bf16(tokens, cols, 2.0, 1, dev, 16), bf16(tokens, cols, 1.0, 2, dev, 0)
    dh = bf16(tokens, cols, 1e-3, 3, dev, 32)
    if tokens > 3:
        dh[2] = 0           # a token without a gradient: zero blocks
        up[3] = 0
    dg, du, tg, tu = swiglu_bwd(f64(dh), f64(gate), f64(up))
    got = pf.puro_fp8_swiglu_bwd_quant_dual(dh, gate, up, transpose_out=transpose_out, pow2=pow2)
    torch.cuda.synchronize()
    for X, T, o, what in ((dg, tg, got[0], "dgate"), (du, tu, got[1], "dup")):
        check_dual(X, T, *o, what, transpose_out, pow2)
    if cols % 128 == 0:
        j = pf.puro_fp8_swiglu_bwd_quant_dual(dh, gate, up, transpose_out=transpose_out, joined=True, pow2=pow2)
        torch.cuda.synchronize()
        ax = 0 if transpose_out else 1
        for k in range(4):
            assert torch.equal(j[k], torch.cat((got[0][k], got[1][k]), ax if k >= 2 else 1))
    else:
        with pytest.raises(ValueError, match="multiple of 128"):
            pf.puro_fp8_swiglu_bwd_quant_dual(dh, gate, up, joined=True)


def test_every_finite_gate(dev):
    """All finite BF16 gate values, subnormal to the largest, with |dh|, |up| <= 1."""
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    bits[(bits & 0x7F80) == 0x7F80] = 0
    gate = torch.from_numpy(bits.reshape(256, 256).view(np.int16)).view(torch.bfloat16).to(dev)
    up = bf16(256, 256, 0.5, 5, dev).clamp(-1, 1)
    dh = bf16(256, 256, 0.5, 6, dev).clamp(-1, 1)
    got = pf.puro_fp8_swiglu_bwd_quant_dual(dh, gate, up)
    torch.cuda.synchronize()
    dg, du, tg, tu = swiglu_bwd(f64(dh), f64(gate), f64(up))
    check_dual(dg, tg, *got[0], "dgate")
    check_dual(du, tu, *got[1], "dup")


def test_halves_of_one_product_and_tiny_gradients(dev):
    tokens, cols = 200, 256
    gu = bf16(tokens, 2 * cols, 1.0, 7, dev)
    for mag in (1.0, 1e-34, 1e-38, 2e-40):
        dh = (torch.randn((tokens, cols), generator=torch.Generator().manual_seed(8)).double() * mag).float()
        dh = dh.bfloat16().to(dev)
        got = pf.puro_fp8_swiglu_bwd_quant_dual(dh, gu[:, :cols], gu[:, cols:])
        torch.cuda.synchronize()
        dg, du, tg, tu = swiglu_bwd(f64(dh), f64(gu[:, :cols]), f64(gu[:, cols:]))
        check_dual(dg, tg, *got[0], "dgate %g" % mag)
        check_dual(du, tu, *got[1], "dup %g" % mag)


def test_no_tokens(dev):
    x = torch.empty((0, 256), dtype=torch.bfloat16, device=dev)
    got = pf.puro_fp8_swiglu_bwd_quant_dual(x, x, x, joined=True)
    assert got[0].shape == (0, 512) and got[2].shape == (512, 0)
