"""puro_fp8_attention and its gradient over a million sequences, nearly all of them empty."""
import pytest
import torch

import attn_ref as ref
import blockwise_fp8_gemm_amd as pf

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,hq,hk", [(64, 64, 1), (128, 33, 1), (64, 34, 2)])
def test_a_million_sequences(dev, dim, hq, hk):
    """2^20 and some sequences: with 64 heads on 1 the gradient's first pass has more than 2^24 workgroups."""
    total = 2 ** 20 + 3
    gen = torch.Generator().manual_seed(hq)
    # sequences that have rows: the first and last ones, the second 2^19's, and some between
    at = sorted({0, 1, 2 ** 19, 2 ** 19 + 1, total - 2, total - 1, *torch.randint(0, total, (30,), generator=gen).tolist()})
    ql, kl = torch.zeros((total,), dtype=torch.int64), torch.zeros((total,), dtype=torch.int64)
    for i, s in enumerate(at):
        ql[s], kl[s] = 1 + i % 2, 2 + (3 * i) % 5
    qo, ko = (torch.cat((torch.zeros((1,), dtype=torch.int64), torch.cumsum(t, 0))) for t in (ql, kl))
    tq, tk = int(qo[-1]), int(ko[-1])
    q, do = ref.bf16(gen, tq, hq * dim, 1.0, 0, dev), ref.bf16(gen, tq, hq * dim, 1e-3, 0, dev)
    k, v = ref.bf16(gen, tk, hk * dim, 1.0, 0, dev), ref.bf16(gen, tk, hk * dim, 1.0, 0, dev)
    plan = (dim, qo.to(torch.int32).to(dev), ko.to(torch.int32).to(dev), 2, 6)
    o, lse = pf.puro_fp8_attention(q, k, v, *plan)
    got = pf.puro_fp8_attention_bwd(do, q, k, v, o, lse, *plan)
    torch.cuda.synchronize()
    qs, ks = ([slice(int(t[s]), int(t[s + 1])) for s in at] for t in (qo, ko))
    want, tol, wl, lt = ref.attention(q, k, v, dim, qs, ks, dim ** -0.5, True)
    ref.close_bf16(o, want, tol, "o")
    assert bool(((ref.f64(lse) - wl).abs() <= lt).all())
    for g, (w, t), what in zip(got, ref.attention_bwd(do, q, k, v, o, lse, dim, qs, ks, dim ** -0.5, True), ("dq", "dk", "dv")):
        ref.close_bf16(g, w, t, what)
