"""The activation gradient's distance from 64 bits, beside that of the same formula in elementary FP32
operations (exp, an IEEE division)."""
import numpy as np
import pytest
import torch

import blockwise_fp8_gemm_amd as pf
from fused_ref import check_dual, f64, swiglu_bwd

pytestmark = pytest.mark.gpu


def gates(lo, hi):
    bits = torch.from_numpy(np.arange(65536, dtype=np.uint32).astype(np.uint16).view(np.int16))
    g = bits.view(torch.bfloat16)
    return g[(g.float() > lo) & (g.float() < hi) & (g.float().abs() > 2.0 ** -10)]


@pytest.mark.parametrize("lo,hi", [(-86.0, -17.0), (-8.0, -2.0), (0.0, 8.0)])
def test_no_further_than_elementary_fp32(dev, lo, hi):
    """One element other than zero per block, so that s_row is |value| / 448, rounded once.

    In units of the mean square of one FP32 rounding, an elementary result has at least 4 (exp, which is rounded
    nearly correctly; g sg; its product with dh; s).  The kernel's exp is one step off at most (4) with a
    correction of its own (1), its reciprocal's correction adds one: at most 9 where the other has 4 at least.
    The root of the mean squares may be 1.5 times as large."""
    g = gates(lo, hi)
    gen = torch.Generator().manual_seed(1)
    tokens, cols = 64, 128 * g.numel()
    gate, dh = (torch.zeros((tokens, cols), dtype=torch.bfloat16) for _ in range(2))
    gate[:, ::128] = g
    # large enough that no result is subnormal (e^-86 = 2^-124)
    dh[:, ::128] = (torch.randn((tokens, g.numel()), generator=gen) * 2.0 ** 40).to(torch.bfloat16)
    up = torch.ones_like(gate)
    dgate, dup = pf.puro_fp8_swiglu_bwd_quant_dual(dh.to(dev), gate.to(dev), up.to(dev))
    torch.cuda.synchronize()
    d32, g32 = dh[:, ::128].float(), g.float()
    e = torch.exp(-g32.abs())
    i = 1 / (1 + e)
    sig, nsig = (torch.where(g32 < 0, a, b) for a, b in ((e * i, i), (i, e * i)))
    x, y = g.double(), dh[:, ::128].double()
    for s, plain, want in ((dup[1], d32 * (g32 * sig), y * x * torch.sigmoid(x)),
                           (dgate[1], d32 * (sig * (1 + g32 * nsig)),
                            y * torch.sigmoid(x) * (1 + x * torch.sigmoid(-x)))):
        some = (want.abs() > 0) & ((x + 1.2785).abs() > 0.3)     # away from the zero of silu'
        rel = [float((((v - want.abs()) / want.abs())[some]).square().mean().sqrt()) * 2 ** 24
               for v in (448 * f64(s), 448 * (plain.abs() / 448).double())]
        assert rel[0] <= 1.5 * rel[1], rel


def test_largest_products(dev):
    """|dh up| up to FP32's largest is what the header asks for: gates small and large beside it."""
    tokens, cols = 40, 256
    gen = torch.Generator().manual_seed(2)
    dh = (torch.rand((tokens, cols), generator=gen) + 1) * 2.0 ** 64
    up = (torch.rand((tokens, cols), generator=gen) + 1) * 2.0 ** 60
    gate = torch.randn((tokens, cols), generator=gen) * torch.tensor([0.01, 1.0, 30.0, 1e9]).repeat(10)[:, None]
    dh, up, gate = (t.to(torch.bfloat16) for t in (dh, up, gate))
    got = pf.puro_fp8_swiglu_bwd_quant_dual(dh.to(dev), gate.to(dev), up.to(dev))
    torch.cuda.synchronize()
    dg, du, tg, tu = swiglu_bwd(f64(dh), f64(gate), f64(up))
    # the products with gate pass FP32's range, the results do not
    assert float((dh.double() * up.double() * gate.double()).abs().max()) > 3.5e38 > 2 * float(dg.abs().max())
    check_dual(dg, tg, *got[0], "dgate")
    check_dual(du, tu, *got[1], "dup")
