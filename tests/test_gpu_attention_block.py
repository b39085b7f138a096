"""An attention block's whole training step through the library: residual sum and norm, joint q/k/v product, head
norms and rotation, attention, output product, and backwards to the block's input gradient and every weight
gradient; and the same weights serving a prompt in two chunks and then single tokens out of padded caches.

Each stage is checked against the 64-bit result of its own inputs as the stage before left them."""
import pytest
import torch

import attn_ref as ref
import blockwise_fp8_gemm_amd as pf
from fused_ref import bf16, check_dual, f64, norm, norm_bwd
from test_gpu_block_step import check_product, rows, tiles

pytestmark = pytest.mark.gpu

EPS = 1e-6


def frequencies(dim, dev):
    return (1e6 ** (-torch.arange(dim // 2, dtype=torch.float64) / (dim // 2))).float().to(dev)


@pytest.mark.parametrize("lens,hq,hk,dim,interleaved", [([130, 1, 77], 4, 2, 128, False), ([64, 200, 3], 6, 2, 64, True)])
def test_training_step(dev, lens, hq, hk, dim, interleaved):
    hidden, tokens = 256, sum(lens)
    cq, ck = hq * dim, hk * dim
    cols = cq + 2 * ck
    gen = torch.Generator().manual_seed(7)
    x, res = bf16(tokens, hidden, 1.0, 1, dev), bf16(tokens, hidden, 2.0, 2, dev)
    w = (1 + 0.1 * torch.randn((hidden,), generator=gen)).to(dev)
    wq, wk = ((1 + 0.1 * torch.randn((dim,), generator=gen)).to(dev) for _ in range(2))
    wqkv = (torch.randn((cols, hidden), generator=gen) * 0.1).to(dev)
    wo = (torch.randn((hidden, cq), generator=gen) * 0.1).to(dev)
    dy = bf16(tokens, hidden, 1e-3, 3, dev)
    pos = ref.i32([i for n in lens for i in range(n)], dev)
    off, freq = ref.i32(ref.offsets(lens), dev), frequencies(dim, dev)
    plan, turn = (dim, off, off, max(lens), max(lens)), (dim, pos, freq)

    (qa, sa, qat, sat), (qo, so, qot, sot) = pf.puro_fp8_quant_weight_grouped([wqkv, wo], transposed=True)
    # forward
    z, rstd, _, qn, sn, qnt, snt = pf.puro_fp8_rmsnorm_quant_dual(x, w, res, eps=EPS)
    joint = pf.puro_fp8_gemm("NT", qn, sn, qa, sa)
    hq_, hk_, hv_ = joint[:, :cq], joint[:, cq:cq + ck], joint[:, cq + ck:]
    q, k, hr = pf.puro_fp8_qk_norm_rope(hq_, hk_, *turn, wq, wk, EPS, interleaved=interleaved)
    o, lse = pf.puro_fp8_attention(q, k, hv_, *plan)
    qh, sh, qht, sht = pf.puro_fp8_quant_dual(o)
    y = pf.puro_fp8_gemm("NT", qh, sh, qo, so)
    # backward
    qy, sy, qyt, syt = pf.puro_fp8_quant_dual(dy)
    dwo = pf.puro_fp8_gemm("NT", qyt, syt, qht, sht, bgran="1x128", out_dtype=torch.float32)
    do = pf.puro_fp8_gemm("NT", qy, sy, qot, sot)
    dq, dk, dv = pf.puro_fp8_attention_bwd(do, q, k, hv_, o, lse, *plan)
    dj, dwq, dwk, qg, sg, qgt, sgt = pf.puro_fp8_qk_norm_rope_bwd_quant_dual(
        dq, dk, dv, hq_, hk_, *turn, hr, wq, wk, interleaved=interleaved, store_dx=True)
    dwa = pf.puro_fp8_gemm("NT", qgt, sgt, qnt, snt, bgran="1x128", out_dtype=torch.float32)
    dn = pf.puro_fp8_gemm("NT", qg, sg, qat, sat)
    dx, dw, *_ = pf.puro_fp8_rmsnorm_bwd_quant_dual(dn, z, rstd, w, dres=dy)
    torch.cuda.synchronize()

    n, tol, _, _ = norm(f64(z), f64(w), EPS)
    check_dual(n, tol, qn, sn, qnt, snt, "norm")
    check_product(joint, rows(qn, sn), tiles(qa, sa), "q/k/v")
    p64, f64s = f64(pos), f64(freq)
    for got, src, wt, heads, what in ((q, hq_, wq, slice(0, hq), "q"), (k, hk_, wk, slice(hq, hq + hk), "k")):
        want, tol, r, rel = ref.rope(f64(src).view(tokens, -1, dim), f64(wt), EPS, p64, f64s, 1.0, interleaved)
        ref.close_bf16(got, want.flatten(1), tol.flatten(1), what)
        assert bool(((f64(hr)[:, heads] - r).abs() <= rel * r).all())
    spans = ref.spans(ref.offsets(lens), None)
    want, tol, _, _ = ref.attention(q, k, hv_, dim, spans, spans, dim ** -0.5, True)
    ref.close_bf16(o, want, tol, "o")
    check_dual(f64(o), torch.zeros_like(f64(o)), qh, sh, qht, sht, "o's codes")
    check_product(y, rows(qh, sh), tiles(qo, so), "y")
    check_product(dwo, rows(qyt, syt), rows(qht, sht), "output weight's gradient")
    check_product(do, rows(qy, sy), tiles(qot, sot), "o's gradient")
    bounds = ref.attention_bwd(do, q, k, hv_, o, lse, dim, spans, spans, dim ** -0.5, True)
    for got, (want, tol), what in zip((dq, dk, dv), bounds, ("dq", "dk", "dv")):
        ref.close_bf16(got, want, tol, what)
    parts = []
    for dy_, src, wt, heads, dwt in ((dq, hq_, wq, slice(0, hq), dwq), (dk, hk_, wk, slice(hq, hq + hk), dwk)):
        want, tol, ew, tw = ref.rope_bwd(f64(dy_).view(tokens, -1, dim), f64(src).view(tokens, -1, dim), f64(hr)[:, heads], f64(wt),
                                         p64, f64s, 1.0, interleaved)
        parts.append((want.flatten(1), tol.flatten(1)))
        assert bool(((f64(dwt) - ew).abs() <= tw).all())
    want = torch.cat((parts[0][0], parts[1][0], f64(dv)), 1)
    tol = torch.cat((parts[0][1], parts[1][1], torch.zeros_like(f64(dv))), 1) + 2.0 ** -147
    ref.close_bf16(dj, want, tol, "joint gradient")
    check_dual(want, tol, qg, sg, qgt, sgt, "joint gradient's codes")
    check_product(dwa, rows(qgt, sgt), rows(qnt, snt), "q/k/v weight's gradient")
    check_product(dn, rows(qg, sg), tiles(qat, sat), "norm's gradient")
    ex, tx, ew, tw = norm_bwd(f64(dn), f64(z), f64(rstd), f64(w), f64(dy))
    ref.close_bf16(dx, ex, tx, "dx")
    assert bool(((f64(dw) - ew).abs() <= tw).all())


def test_serving(dev):
    """A prompt in two chunks and ten single tokens over padded caches: every row is the whole prompt's."""
    hq, hk, dim, cap = 4, 2, 128, 200
    lens = [150, 97]
    gen = torch.Generator().manual_seed(8)
    joint = [ref.bf16(gen, n, (hq + 2 * hk) * dim, 1.0, 0, dev) for n in lens]
    wq, wk = ((1 + 0.1 * torch.randn((dim,), generator=gen)).to(dev) for _ in range(2))
    freq, cq, ck = frequencies(dim, dev), hq * dim, hk * dim
    kc, vc = (torch.full((2 * cap, ck), float("nan"), dtype=torch.bfloat16, device=dev) for _ in range(2))
    whole, outs, filled = [], [[], []], [0, 0]
    for x, n in zip(joint, lens):
        off = ref.i32([0, n], dev)
        q, k, _ = pf.puro_fp8_qk_norm_rope(x[:, :cq], x[:, cq:cq + ck], dim, ref.i32(list(range(n)), dev), freq, wq, wk)
        whole.append(pf.puro_fp8_attention(q, k, x[:, cq + ck:], dim, off, off, n, n))

    def step(counts):
        """counts new rows of each sequence, appended to the caches and attended."""
        part = torch.cat([x[f:f + c] for x, f, c in zip(joint, filled, counts)])
        pos = [f + i for f, c in zip(filled, counts) for i in range(c)]
        q, k, _ = pf.puro_fp8_qk_norm_rope(part[:, :cq], part[:, cq:cq + ck], dim, ref.i32(pos, dev), freq, wq, wk, store_rstd=False)
        at = torch.tensor([s * cap + p for s, c in enumerate(counts) for p in range(filled[s], filled[s] + c)], device=dev)
        kc[at], vc[at] = k, part[:, cq + ck:]
        for s, c in enumerate(counts):
            filled[s] += c
        o, lse = pf.puro_fp8_attention(q, kc, vc, dim, ref.i32(ref.offsets(counts), dev), ref.i32([0, cap], dev), max(counts), cap,
                                       k_lengths=ref.i32(filled, dev))
        a = 0
        for s, c in enumerate(counts):
            outs[s].append((o[a:a + c], lse[:, a:a + c]))
            a += c

    step([100, 40])
    step([40, 47])
    for _ in range(10):
        step([1, 1])
    torch.cuda.synchronize()
    for s, n in enumerate(lens):
        assert filled[s] == n
        o, lse = torch.cat([a for a, _ in outs[s]]), torch.cat([b for _, b in outs[s]], 1)
        # the same rows by other orders of the same sums: each within its bound of the exact row
        want, tol, wl, lt = ref.attention(*[t[s * cap:s * cap + n] if t.shape[0] == 2 * cap else t for t in (
            torch.cat([pf.puro_fp8_qk_norm_rope(joint[s][:, :cq], joint[s][:, cq:cq + ck], dim, ref.i32(list(range(n)), dev),
                                                freq, wq, wk)[0]]), kc, vc)], dim, [slice(0, n)], [slice(0, n)], dim ** -0.5, True)
        ref.close_bf16(o, want, tol, "chunks")
        ref.close_bf16(whole[s][0], want, tol, "whole")
        assert bool(((ref.f64(lse) - wl).abs() <= lt).all()) and bool(((ref.f64(whole[s][1]) - wl).abs() <= lt).all())
