"""The norm, activation-gradient and orthogonalisation calls captured in HIP graphs, on side streams,
from several host threads at once, and with a workspace handed from call to call."""
import threading

import pytest
import torch

import blockwise_fp8_gemm_amd as pf
from fused_ref import bf16

pytestmark = pytest.mark.gpu


def inputs(dev, seed, tokens=300, cols=640):
    gen = torch.Generator().manual_seed(seed)
    return {"x": bf16(tokens, cols, 1.0, seed, dev), "res": bf16(tokens, cols, 2.0, seed + 1, dev),
            "dy": bf16(tokens, cols, 1e-3, seed + 2, dev), "w": (1 + torch.rand((cols,), generator=gen)).to(dev),
            "g": [torch.randn((256, 384), generator=gen).to(dev), torch.randn((300, 160), generator=gen).to(dev)]}


def calls(d, **kw):
    """Every entry point once; all outputs."""
    a = pf.puro_fp8_rmsnorm_quant_act(d["x"], d["w"], d["res"], store_h=True, **kw)
    b = pf.puro_fp8_rmsnorm_quant_dual(d["x"], d["w"], d["res"], store_h=True, **kw)
    c = pf.puro_fp8_rmsnorm_bwd_quant_dual(d["dy"], b[0], b[1], d["w"], d["res"], **kw)
    e = pf.puro_fp8_swiglu_bwd_quant_dual(d["dy"], d["x"], d["res"], joined=True, **kw)
    f = pf.puro_fp8_swiglu_bwd_quant_dual(d["dy"], d["x"], d["res"], transpose_out=False, pow2=True, **kw)
    o = pf.puro_fp8_newton_schulz_grouped(d["g"], **kw)
    return [*a, *b, *c, *e, *f[0], *f[1], *o]


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def test_graph_replays(dev):
    d = inputs(dev, 10)
    ref = [t.clone() for t in calls(d)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls(d)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls(d)
    for k in range(4):
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, ref), k
        assert same(calls(d), ref), k       # eager work between the replays
    # new inputs in the captured buffers
    e = inputs(dev, 20)
    for key in ("x", "res", "dy", "w"):
        d[key].copy_(e[key])
    for p, q in zip(d["g"], e["g"]):
        p.copy_(q)
    graph.replay()
    torch.cuda.synchronize()
    assert same(out, calls(e))


def test_two_graphs_with_workspaces_of_their_own(dev):
    """Two captured graphs in flight on two streams."""
    ds = [inputs(dev, 30), inputs(dev, 40)]
    refs = [[t.clone() for t in calls(d)] for d in ds]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for d in ds:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(calls(d))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert same(outs[0], refs[0]) and same(outs[1], refs[1])


def test_side_streams(dev):
    """Work launched on other streams than the current one, while the current one allocates."""
    ds = [inputs(dev, 50 + k) for k in range(3)]
    refs = [[t.clone() for t in calls(d)] for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    for _ in range(3):
        outs = []
        for s, d in zip(streams, ds):
            outs.append(calls(d, stream=s))
            torch.empty((1 << 20,), device=dev).fill_(float("nan"))
        torch.cuda.synchronize()
        for o, r in zip(outs, refs):
            assert same(o, r)


def test_host_threads(dev):
    ds = [inputs(dev, 70 + k) for k in range(4)]
    refs = [[t.clone() for t in calls(d)] for d in ds]
    torch.cuda.synchronize()
    bad = []

    def work(k):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(4):
                    out = calls(ds[k])
                    s.synchronize()
                    if not same(out, refs[k]):
                        bad.append(k)
        except Exception as e:   # reported by the main thread
            bad.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


def test_one_workspace_from_call_to_call(dev):
    """A workspace given to calls that follow each other on a stream; what it held does not matter."""
    a, b = inputs(dev, 90), inputs(dev, 95, tokens=129, cols=384)
    ws = torch.full((1 << 24,), 0xFF, dtype=torch.uint8, device=dev)
    for d in (a, b, a):
        z, r = pf.puro_fp8_rmsnorm_quant_dual(d["x"], d["w"], d["res"])[:2]
        ref = pf.puro_fp8_rmsnorm_bwd_quant_dual(d["dy"], z, r, d["w"])
        assert same(pf.puro_fp8_rmsnorm_bwd_quant_dual(d["dy"], z, r, d["w"], workspace=ws), ref)
        ref = pf.puro_fp8_newton_schulz_grouped(d["g"])
        assert same(pf.puro_fp8_newton_schulz_grouped(d["g"], workspace=ws), ref)


def test_overlapping_reads_are_allowed(dev):
    """One tensor in several input places, and one matrix twice in a call."""
    d = inputs(dev, 99)
    x, g = d["x"], d["g"][0]
    a = pf.puro_fp8_rmsnorm_quant_dual(x, d["w"], x)
    b = pf.puro_fp8_rmsnorm_quant_dual(x, d["w"], x.clone())
    assert same([t for t in a if t is not None], [t for t in b if t is not None])
    u, v = pf.puro_fp8_newton_schulz_grouped([g, g])
    assert torch.equal(u, v) and torch.equal(u, pf.puro_fp8_newton_schulz_grouped([g])[0])
