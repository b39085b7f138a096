"""The gradient of attention where a row of many keys has its weight on a few of them, against the formula with the
exact o.  Such rows form D from o as the forward left it, rounded to BF16: half a step of every term of do . o, where dP
and D nearly cancel."""
import pytest
import torch

import attn_ref as ref
import blockwise_fp8_gemm_amd as pf

pytestmark = pytest.mark.gpu


def bounds(do, q, k, v, o, lse, scale, causal):
    """head_bwd with the exact o, and dq's and dk's bounds with that much more in D."""
    dq, dk, dv, tq, tk, tv = ref.head_bwd(q, k, v, do, o, lse, scale, causal)
    hide = ref.hidden(q.shape[0], k.shape[0], causal)
    p = torch.where(hide, 0.0, torch.exp(scale * (q @ k.t()) - lse[:, None]))
    more = p * ref.B * (do * o).abs().sum(1, keepdim=True) * (1 + ref.B)
    return (dq, tq + scale * more @ k.abs()), (dk, tk + scale * more.t() @ q.abs()), (dv, tv)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,m", [(300, 300), (70, 1000)])
@pytest.mark.parametrize("std", [1.0, 3.0, 6.0])
def test_against_the_exact_output(dev, std, n, m, causal, dim):
    gen = torch.Generator().manual_seed(n + int(std))
    q, do = ref.bf16(gen, n, dim, std, 0, dev), ref.bf16(gen, n, dim, 1e-3, 0, dev)
    k, v = ref.bf16(gen, m, dim, std, 0, dev), ref.bf16(gen, m, dim, 1.0, 0, dev)
    scale = dim ** -0.5
    o, _, lse, _, _, _ = ref.head(ref.f64(q), ref.f64(k), ref.f64(v), scale, causal)
    lse = lse.float()
    got = pf.puro_fp8_attention_bwd(do, q, k, v, o.to(torch.bfloat16).to(dev), lse[None].to(dev), dim, ref.i32([0, n], dev),
                                    ref.i32([0, m], dev), n, m, causal=causal)
    torch.cuda.synchronize()
    want = bounds(ref.f64(do), ref.f64(q), ref.f64(k), ref.f64(v), o, ref.f64(lse), scale, causal)
    for g, (w, t), what in zip(got, want, ("dq", "dk", "dv")):
        g = ref.f64(g)
        off = (g - w).abs() - (t + ref.B * (w.abs() + t) + 2.0 ** -134)
        assert bool((off <= 0).all()), (what, float(off.max()))
