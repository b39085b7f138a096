"""The attention and head-norm calls captured in HIP graphs, on side streams, from several host threads at once, and
with a workspace handed from call to call."""
import threading

import pytest
import torch

import attn_ref as ref
import blockwise_fp8_gemm_amd as pf

pytestmark = pytest.mark.gpu

HQ, HK, DIM = 4, 2, 64
LENS, MANY = [70, 5, 200], [700, 90, 2300]


def inputs(dev, seed):
    gen = torch.Generator().manual_seed(seed)
    t, n = sum(LENS), sum(MANY)
    d = {"q": ref.bf16(gen, t, HQ * DIM, 1.0, 0, dev), "k": ref.bf16(gen, t, HK * DIM, 1.0, 0, dev),
         "v": ref.bf16(gen, t, HK * DIM, 1.0, 0, dev), "do": ref.bf16(gen, t, HQ * DIM, 1e-3, 0, dev),
         "one": ref.bf16(gen, len(MANY), HQ * DIM, 1.0, 0, dev), "kc": ref.bf16(gen, n, HK * DIM, 1.0, 0, dev),
         "vc": ref.bf16(gen, n, HK * DIM, 1.0, 0, dev), "w": (1 + torch.rand((2, DIM), generator=gen)).to(dev),
         "off": ref.i32(ref.offsets(LENS), dev), "ones": ref.i32(ref.offsets([1] * len(MANY)), dev),
         "many": ref.i32(ref.offsets(MANY), dev), "pos": torch.randint(0, 9999, (t,), generator=gen).to(torch.int32).to(dev),
         "freq": (1e4 ** (-torch.arange(DIM // 2) / (DIM // 2))).to(dev)}
    return d


def calls(d, **kw):
    """Every entry point once, each on the results of the one before; all outputs."""
    q, k, rstd = pf.puro_fp8_qk_norm_rope(d["q"], d["k"], DIM, d["pos"], d["freq"], d["w"][0], d["w"][1], **kw)
    plan = (DIM, d["off"], d["off"], max(LENS), max(LENS))
    o, lse = pf.puro_fp8_attention(q, k, d["v"], *plan, **kw)
    dq, dk, dv = pf.puro_fp8_attention_bwd(d["do"], q, k, d["v"], o, lse, *plan, **kw)
    g = pf.puro_fp8_qk_norm_rope_bwd_quant_dual(dq, dk, dv, d["q"], d["k"], DIM, d["pos"], d["freq"], rstd, d["w"][0],
                                                d["w"][1], store_dx=True, **kw)
    one = pf.puro_fp8_attention(d["one"], d["kc"], d["vc"], DIM, d["ones"], d["many"], 1, max(MANY), **kw)   # split
    return [q, k, rstd, o, lse, dq, dk, dv, *g, *one]


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def test_graph_replays(dev):
    d = inputs(dev, 10)
    ref_out = [t.clone() for t in calls(d)]
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
        assert same(out, ref_out), k
        assert same(calls(d), ref_out), k       # eager work between the replays
    # new inputs in the captured buffers, and other lengths inside the captured maxima
    e = inputs(dev, 20)
    e["off"], e["many"] = ref.i32([0, 60, 130, 275], dev), ref.i32([0, 10, 2300, 3090], dev)
    for key in d:
        d[key].copy_(e[key])
    graph.replay()
    torch.cuda.synchronize()
    assert same(out, calls(e))


def test_two_graphs_in_flight(dev):
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


def test_workspaces_are_checked(dev):
    d = inputs(dev, 90)
    args = (d["one"], d["kc"], d["vc"], DIM, d["ones"], d["many"], 1, max(MANY))
    want = pf.puro_fp8_attention(*args)
    need = pf.puro_fp8_attention_workspace_size(HQ, HK, DIM, len(MANY), len(MANY), sum(MANY), 1, max(MANY))
    assert need > 0
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=dev)
    for _ in range(2):
        assert same(pf.puro_fp8_attention(*args, workspace=ws), want)
    with pytest.raises(pf.PuroError):
        pf.puro_fp8_attention(*args, workspace=ws[:need - 1])
    for bad in (torch.empty((1 << 20,), dtype=torch.uint8), torch.empty((1 << 21,), dtype=torch.uint8, device=dev)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            pf.puro_fp8_attention(*args, workspace=bad)
    with pytest.raises(ValueError, match="k_offsets"):
        pf.puro_fp8_attention(d["one"], d["kc"], d["vc"], DIM, d["ones"], d["many"].cpu(), 1, max(MANY))
    with pytest.raises(ValueError, match="sequences"):
        pf.puro_fp8_attention(d["one"], d["kc"], d["vc"], DIM, d["ones"], d["many"][:2], 1, max(MANY))
