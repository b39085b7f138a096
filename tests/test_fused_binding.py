"""Binding of the norm, activation-gradient and orthogonalisation calls: every argument by name, workspaces
that are not the GPU's refused on the host, and the residual sum in place."""
import pytest
import torch

import blockwise_fp8_gemm_amd as pf
from fused_ref import bf16


def test_first_argument_by_name():
    x, w = torch.zeros((4, 128), dtype=torch.bfloat16), torch.ones((128,))
    for call in (lambda: pf.puro_fp8_rmsnorm_quant_act(x=x, weight=w),
                 lambda: pf.puro_fp8_rmsnorm_quant_dual(weight=w, x=x),
                 lambda: pf.puro_fp8_rmsnorm_bwd_quant_dual(dy=x, z=x, rstd=torch.ones((4,)), weight=w),
                 lambda: pf.puro_fp8_swiglu_bwd_quant_dual(dh=x, gate=x, up=x),
                 lambda: pf.puro_fp8_newton_schulz_grouped(grads=[x])):
        with pytest.raises(ValueError, match="on the GPU"):
            call()
    assert pf.puro_fp8_newton_schulz_grouped(grads=[]) == []


def test_workspace_of_another_device_is_refused():
    gpu = torch.device("cuda", 0)
    with pytest.raises(ValueError, match="workspace"):
        pf._workspace(torch.empty((1 << 20,), dtype=torch.uint8), lambda: 0, gpu)


@pytest.mark.gpu
def test_workspace_is_checked(dev):
    x, w = bf16(40, 200, 1.0, 1, dev), torch.ones((200,), device=dev)
    need = pf.puro_fp8_rmsnorm_bwd_workspace_size(40, 200)
    rstd = torch.ones((40,), device=dev)
    g = torch.randn((64, 80), device=dev)
    for bad in (torch.empty((1 << 22,), dtype=torch.uint8), torch.empty((1 << 23,), dtype=torch.uint8, device=dev)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            pf.puro_fp8_rmsnorm_bwd_quant_dual(x, x, rstd, w, workspace=bad)
        with pytest.raises(ValueError, match="workspace"):
            pf.puro_fp8_newton_schulz_grouped([g], workspace=bad)
    small = torch.empty((need - 1,), dtype=torch.uint8, device=dev)
    with pytest.raises(pf.PuroError):
        pf.puro_fp8_rmsnorm_bwd_quant_dual(x, x, rstd, w, workspace=small)
    a = pf.puro_fp8_rmsnorm_bwd_quant_dual(dy=x, z=x, rstd=rstd, weight=w)
    b = pf.puro_fp8_rmsnorm_bwd_quant_dual(x, x, rstd, w,
                                           workspace=torch.empty((need,), dtype=torch.uint8, device=dev))
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,cols", [(1, 1), (300, 1000), (5000, 129), (3, 20000), (2100, 8200)])
@pytest.mark.parametrize("over", ["x", "residual"])
def test_sum_in_place(dev, tokens, cols, over):
    """z over x or over the residual: the bits of the call with a z of its own."""
    x, res = bf16(tokens, cols, 1.0, 2, dev, 16), bf16(tokens, cols, 2.0, 3, dev)
    w = torch.ones((cols,), device=dev)
    for call in (pf.puro_fp8_rmsnorm_quant_act, pf.puro_fp8_rmsnorm_quant_dual):
        want = call(x, w, res, store_h=True)
        # as they lie: the same row strides, so that z has its operand's
        a, b = bf16(tokens, cols, 1.0, 2, dev, 16), bf16(tokens, cols, 2.0, 3, dev)
        z = a if over == "x" else b
        got = call(a, w, b, z=z, store_h=True)
        torch.cuda.synchronize()
        assert got[0].data_ptr() == z.data_ptr()
        assert all(torch.equal(p, q) for p, q in zip(want, got))
        assert torch.equal(b if over == "x" else a, res if over == "x" else x)
