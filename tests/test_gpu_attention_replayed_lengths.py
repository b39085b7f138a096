"""Attention and its gradient captured once, replayed over lengths that change between the replays: shorter, empty, and
longer than the maxima of the capture (each replay against an eager call on the same arrays and the 64-bit formula)."""
import pytest
import torch

import attn_ref as ref
import blockwise_fp8_gemm_amd as pf

pytestmark = pytest.mark.gpu

HQ, HK, CAP, MAX_Q, MAX_K = 4, 2, 400, 60, 300


@pytest.mark.parametrize("dim", [64, 128])
def test_replays(dev, monkeypatch, dim):
    gen = torch.Generator().manual_seed(dim)
    n = 3
    q, do = ref.bf16(gen, n * CAP, HQ * dim, 1.0, 0, dev), ref.bf16(gen, n * CAP, HQ * dim, 1e-3, 0, dev)
    k, v = ref.bf16(gen, n * CAP, HK * dim, 1.0, 0, dev), ref.bf16(gen, n * CAP, HK * dim, 1.0, 0, dev)
    starts = [i * CAP for i in range(n)]
    off, ql, kl = ref.i32(starts, dev), ref.i32([1] * n, dev), ref.i32([1] * n, dev)
    nan = [torch.full_like(t, float("nan")) for t in (q, q, k, v)]
    o, dq, dk, dv = nan
    lse = torch.full((HQ, n * CAP), float("nan"), device=dev)
    plan, kw = (dim, off, off, MAX_Q, MAX_K), {"q_lengths": ql, "k_lengths": kl}

    def calls(o, lse, dq, dk, dv):
        pf.puro_fp8_attention(q, k, v, *plan, o=o, lse=lse, **kw)
        pf.puro_fp8_attention_bwd(do, q, k, v, o, lse, *plan, dq=dq, dk=dk, dv=dv, **kw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls(o, lse, dq, dk, dv)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(o, lse, dq, dk, dv)
    for qn, kn in (([60, 1, 33], [300, 1, 33]), ([0, 5, 60], [10, 0, 60]), ([100, 61, 400], [100, 400, 400]), ([400, 7, -1], [350, 301, 5]),
                   ([60, 1, 33], [300, 1, 33])):
        outs = (o, lse, dq, dk, dv)
        for t in outs:
            t.fill_(float("nan"))
        ql.copy_(ref.i32(qn, dev))
        kl.copy_(ref.i32(kn, dev))
        graph.replay()
        torch.cuda.synchronize()
        eager = [torch.full_like(t, float("nan")) for t in outs]
        calls(*eager)
        torch.cuda.synchronize()
        assert all(torch.equal(torch.nan_to_num(a, nan=7.0), torch.nan_to_num(b, nan=7.0)) for a, b in zip(outs, eager)), (qn, kn)
        for i, (a, b) in enumerate(zip(qn, kn)):
            shift = max(b, 0) - max(a, 0)
            monkeypatch.setattr(ref, "hidden", lambda x, y, c, shift=shift: (torch.arange(y) > torch.arange(x)[:, None] + shift) & c)
            rows = slice(starts[i], starts[i] + CAP)
            qs, ks = [slice(0, max(0, min(a, MAX_Q)))], [slice(0, max(0, min(b, MAX_K)))]
            want, tol, wl, lt = ref.attention(q[rows], k[rows], v[rows], dim, qs, ks, dim ** -0.5, True)
            ref.close_bf16(o[rows], want, tol, ("o", qn, kn, i))
            got = ref.f64(lse[:, rows])
            assert torch.equal(torch.isnan(got), torch.isnan(wl)) and torch.equal(torch.isinf(got), torch.isinf(wl))
            fine = torch.isfinite(wl)
            assert bool(((got - wl).abs()[fine] <= lt[fine]).all())
            bounds = ref.attention_bwd(do[rows], q[rows], k[rows], v[rows], o[rows], lse[:, rows], dim, qs, ks, dim ** -0.5, True)
            for g, (w, t), what in zip((dq, dk, dv), bounds, ("dq", "dk", "dv")):
                ref.close_bf16(g[rows], w, t, (what, qn, kn, i))
