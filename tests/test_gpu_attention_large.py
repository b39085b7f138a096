"""Attention and head norms where sizes pass a limit: rows whose byte offsets pass 32 bits, one sequence longer than
that, enough workgroups for every form of the gradient, and many sequences."""
import pytest
import torch

import attn_ref as ref
import blockwise_fp8_gemm_amd as pf
import test_gpu_attention as fwd
import test_gpu_attention_bwd as bwd

pytestmark = pytest.mark.gpu

STRIDE = 4096      # elements of a row of a wide tensor that the head is a part of


def wide(dev, rows, cols):
    return torch.empty((rows, STRIDE), dtype=torch.bfloat16, device=dev)[:, :cols]


@pytest.mark.parametrize("q_len", [1, 40])
def test_sequences_past_4_gb(dev, q_len):
    """Sequences at both ends of a cache of 5 GB, forward and backward."""
    rows, n, dim = 600000, 300, 64
    gen = torch.Generator().manual_seed(1)
    k, v, dk, dv = (wide(dev, rows, dim) for _ in range(4))
    starts = [0, rows - n]
    for s in starts:
        k[s:s + n] = ref.bf16(gen, n, dim, 1.0, 0, dev)
        v[s:s + n] = ref.bf16(gen, n, dim, 1.0, 0, dev)
    q, do = ref.bf16(gen, 2 * q_len, 2 * dim, 1.0, 0, dev), ref.bf16(gen, 2 * q_len, 2 * dim, 1e-3, 0, dev)
    plan = (dim, ref.i32([0, q_len, 2 * q_len], dev), ref.i32(starts, dev), q_len, n)
    lens = ref.i32([n, n], dev)
    o, lse = pf.puro_fp8_attention(q, k, v, *plan, k_lengths=lens)
    got = pf.puro_fp8_attention_bwd(do, q, k, v, o, lse, *plan, k_lengths=lens, dk=dk, dv=dv)
    torch.cuda.synchronize()
    near = [torch.cat([t[s:s + n] for s in starts]) for t in (k, v, dk, dv)]
    qs, ks = [slice(0, q_len), slice(q_len, 2 * q_len)], [slice(0, n), slice(n, 2 * n)]
    want, tol, wl, lt = ref.attention(q, near[0], near[1], dim, qs, ks, 0.125, True)
    ref.close_bf16(o, want, tol, "o")
    fwd.check_lse(lse, wl, lt, "lse")
    bounds = ref.attention_bwd(do, q, near[0], near[1], o, lse, dim, qs, ks, 0.125, True)
    for g, (w, t), what in zip((got[0], near[2], near[3]), bounds, ("dq", "dk", "dv")):
        ref.close_bf16(g, w, t, what)


def test_a_sequence_past_4_gb(dev):
    rows, dim = 600000, 64
    gen = torch.Generator().manual_seed(2)
    k, v = wide(dev, rows, dim), wide(dev, rows, dim)
    k.copy_(ref.bf16(gen, rows, dim, 1.0, 0, dev))
    v.copy_(ref.bf16(gen, rows, dim, 1.0, 0, dev) + 1)
    for q_len in (1, 50):
        q = ref.bf16(gen, q_len, 2 * dim, 1.0, 0, dev)
        o, lse = pf.puro_fp8_attention(q, k, v, dim, ref.i32([0, q_len], dev), ref.i32([0, rows], dev), q_len, rows)
        torch.cuda.synchronize()
        want, tol, wl, lt = ref.attention(q, k, v, dim, [slice(0, q_len)], [slice(0, rows)], 0.125, True)
        ref.close_bf16(o, want, tol, "o")
        # the bound for any order of so many additions is wide; here a lane adds at most 600000 / 64 / 2 terms (64 shares,
        # two lanes a row), 4688 U of the sum, and the mean of |v| is 1.17: half a step for P, half a step of o near one
        assert float((ref.f64(o) - want).abs().max()) <= 2.2 * ref.B and float((ref.f64(lse) - wl).abs().max()) <= 4e-4
        fwd.check_lse(lse, wl, lt, "lse")


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_backward_with_many_workgroups(dev, dim, causal):
    """More workgroups of 128 keys, and of 256 rows, than there are CUs."""
    bwd.run(dev, 64, 64, dim, [520], [520], causal, seed=3)
    bwd.run(dev, 33, 33, dim, [1100], [1037], causal, seed=4)


@pytest.mark.parametrize("dim", [64, 128])
def test_many_sequences(dev, dim):
    gen = torch.Generator().manual_seed(5)
    q = torch.randint(0, 150, (300,), generator=gen).tolist()
    k = [n + int(torch.randint(0, 3, (1,), generator=gen)) for n in q]
    fwd.run(dev, 2, 1, dim, q, k, True, seed=6)
    bwd.run(dev, 2, 1, dim, q, k, True, seed=7)
    ones = [1] * 300
    fwd.run(dev, 4, 2, dim, ones, q, True, seed=8)


def test_rope_rows_past_4_gb(dev):
    tokens, dim = 600000, 64
    gen = torch.Generator().manual_seed(9)
    q, k = wide(dev, tokens, dim), wide(dev, tokens, dim)
    x = ref.bf16(gen, tokens, dim, 1.0, 0, dev)
    q.copy_(x)
    k.copy_(x)
    pos = torch.arange(tokens, device=dev, dtype=torch.int32)
    freq = (1e4 ** (-torch.arange(32, dtype=torch.float64) / 32)).float().to(dev)
    w = torch.ones((dim,), device=dev)
    y, z, rstd = pf.puro_fp8_qk_norm_rope(q, k, dim, pos, freq, w, w, q_out=q)
    torch.cuda.synchronize()
    assert torch.equal(y, z)
    at = torch.cat((torch.arange(100), torch.arange(tokens - 100, tokens)))
    want, tol, _, _ = ref.rope(ref.f64(x[at]).view(200, 1, dim), ref.f64(w), 1e-6, at.double(), ref.f64(freq), 1.0, False)
    ref.close_bf16(y[at], want.flatten(1), tol.flatten(1), "rope")
    d = (y, z, x)
    _, _, _, qr, sr, qt, st = pf.puro_fp8_qk_norm_rope_bwd_quant_dual(*d, x, x, dim, pos, freq, rstd, w, w)
    few = [t[at] for t in d]
    r64 = ref.f64(rstd[at])
    parts = [ref.rope_bwd(ref.f64(t).view(200, 1, dim), ref.f64(x[at]).view(200, 1, dim), r64[:, h:h + 1], ref.f64(w), at.double(),
                          ref.f64(freq), 1.0, False) for h, t in enumerate(few[:2])]
    from fused_ref import check_blocks
    want = torch.cat([p[0].flatten(1) for p in parts] + [ref.f64(few[2])], 1)
    tol = torch.cat([p[1].flatten(1) for p in parts] + [torch.zeros((200, dim), dtype=torch.float64)], 1)
    check_blocks(want, tol, qr[at], sr[at], "codes")


def test_many_sequences_with_loose_maxima(dev):
    """Maxima far above the lengths: most workgroups find nothing to do."""
    lens = [(7 * i) % 90 for i in range(320)]
    fwd.run(dev, 8, 4, 128, lens, lens, True, seed=9, gap=180, loose=1 << 16)
    bwd.run(dev, 8, 4, 128, lens, lens, True, seed=9, gap=180, loose=1 << 16)
