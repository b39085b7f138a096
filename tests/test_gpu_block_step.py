"""A feed-forward block's whole training step through the library: residual sum and norm, gate/up
product, gated activation, down product, and backwards to the block's input gradient, the weight
gradients, their orthogonalised updates and the requantised weights.

Each stage is checked against the 64-bit result of its own inputs as the stage before left them
(codes times scales), so that a layout, a scale or a stride that one call writes and the next reads
differently shows at that link.  GEMM tolerances are those of the GEMM's own tests."""
import pytest
import torch

import blockwise_fp8_gemm_amd as pf
from fused_ref import bf16, check_dual, close_bf16, code_values, f64, norm, norm_bwd, swiglu_bwd
from test_gpu_newton_schulz import check as check_orthogonal

pytestmark = pytest.mark.gpu

EPS = 1e-6


def rows(q, s):
    """Values of a copy in 1x128 blocks along its rows."""
    v = code_values(q)
    return v * f64(s).repeat_interleave(128, 1)[:, :v.shape[1]]


def tiles(q, s):
    v = code_values(q)
    return v * f64(s).repeat_interleave(128, 0)[:v.shape[0]].repeat_interleave(128, 1)[:, :v.shape[1]]


def check_product(C, A, B, what):
    """C against A B^T: 2^-22 of sum |a b| per 128-wide block and four more (FP32 promotion), one BF16 rounding."""
    exact, mag = A @ B.t(), A.abs() @ B.abs().t()
    tol = (A.shape[1] // 128 + 5) * 2.0 ** -23 * mag
    if C.dtype == torch.bfloat16:
        close_bf16(C, exact, tol, what)
    else:
        assert bool(((f64(C) - exact).abs() <= tol).all()), what


@pytest.mark.parametrize("tokens,hidden,ffn", [(256, 256, 384), (200, 384, 256)])
def test_feed_forward_step(dev, tokens, hidden, ffn):
    gen = torch.Generator().manual_seed(5)
    x, res = bf16(tokens, hidden, 1.0, 1, dev), bf16(tokens, hidden, 2.0, 2, dev)
    w = (1 + 0.1 * torch.randn((hidden,), generator=gen)).to(dev)
    wgu = (torch.randn((2 * ffn, hidden), generator=gen) * 0.05).to(dev)      # gate rows, then up rows
    wd = (torch.randn((hidden, ffn), generator=gen) * 0.05).to(dev)
    dy = bf16(tokens, hidden, 1e-3, 3, dev)

    (qgu, sgu, qgut, sgut), (qd, sd, qdt, sdt) = pf.puro_fp8_quant_weight_grouped([wgu, wd], transposed=True)
    # forward
    z, rstd, _, qn, sn, qnt, snt = pf.puro_fp8_rmsnorm_quant_dual(x, w, res, eps=EPS)
    gu = pf.puro_fp8_gemm("NT", qn, sn, qgu, sgu)
    gate, up = gu[:, :ffn], gu[:, ffn:]
    h, qh, sh, qht, sht = pf.puro_fp8_swiglu_quant_dual(gate, up)
    y = pf.puro_fp8_gemm("NT", qh, sh, qd, sd)
    # backward
    qy, sy, qyt, syt = pf.puro_fp8_quant_dual(dy)
    dwd = pf.puro_fp8_gemm("NT", qyt, syt, qht, sht, bgran="1x128", out_dtype=torch.float32)
    dh = pf.puro_fp8_gemm("NT", qy, sy, qdt, sdt)
    qg, sg, qgt, sgt = pf.puro_fp8_swiglu_bwd_quant_dual(dh, gate, up, joined=True)
    dwgu = pf.puro_fp8_gemm("NT", qgt, sgt, qnt, snt, bgran="1x128", out_dtype=torch.float32)
    dn = pf.puro_fp8_gemm("NT", qg, sg, qgut, sgut)
    dx, dw, qx, sx, qxt, sxt = pf.puro_fp8_rmsnorm_bwd_quant_dual(dn, z, rstd, w, dres=dy)
    # update
    od, ogu = pf.puro_fp8_newton_schulz_grouped([dwd, dwgu])
    wgu2, wd2 = wgu - 0.02 * ogu.float(), wd - 0.02 * od.float()
    (qgu2, sgu2), (qd2, sd2) = pf.puro_fp8_quant_weight_grouped([wgu2, wd2])
    torch.cuda.synchronize()

    zx = f64((x.float() + res.float()).bfloat16())
    assert torch.equal(f64(z), zx)
    n, tol, _, _ = norm(zx, f64(w), EPS)
    check_dual(n, tol, qn, sn, qnt, snt, "norm")
    check_product(gu, rows(qn, sn), tiles(qgu, sgu), "gate/up")
    check_dual(f64(h), torch.zeros_like(f64(h)), qh, sh, qht, sht, "activation")
    check_product(y, rows(qh, sh), tiles(qd, sd), "down")
    check_product(dwd, rows(qyt, syt), rows(qht, sht), "down's weight gradient")
    check_product(dh, rows(qy, sy), tiles(qdt, sdt), "activation's gradient")
    dg, du, tg, tu = swiglu_bwd(f64(dh), f64(gate), f64(up))
    check_dual(torch.cat((dg, du), 1), torch.cat((tg, tu), 1), qg, sg, qgt, sgt, "gate/up gradient")
    check_product(dwgu, rows(qgt, sgt), rows(qnt, snt), "gate/up's weight gradient")
    check_product(dn, rows(qg, sg), tiles(qgut, sgut), "norm's gradient")
    ex, tx, ew, tw = norm_bwd(f64(dn), zx, f64(rstd), f64(w), f64(dy))
    close_bf16(dx, ex, tx, "dx")
    check_dual(ex, tx, qx, sx, qxt, sxt, "dx")
    assert bool(((f64(dw) - ew).abs() <= tw).all())
    check_orthogonal(od, dwd)
    check_orthogonal(ogu, dwgu)
    # the requantised weights stand for the updated ones (half a step of E4M3, 2^-4 of a value or 2^-10 s)
    off = (tiles(qgu2, sgu2) - f64(wgu2)).abs() - (2.0 ** -4 * f64(wgu2).abs() + 2.0 ** -10 * float(sgu2.max()))
    assert bool((off <= 1e-9).all())
    assert not torch.equal(qd2, qd)
