"""puro_fp8_attention_bwd against the 64-bit formula and against differences of the 64-bit forward."""
import pytest
import torch

import blockwise_fp8_gemm_amd as pf
import attn_ref as ref

pytestmark = pytest.mark.gpu


def case(dev, hq, hk, dim, q_lens, k_lens, causal, seed=0, scale=None, pad=0, std=1.0, gap=0, loose=0):
    gen = torch.Generator().manual_seed(seed)
    scale = scale or dim ** -0.5
    qo, ko = [sum(q_lens[:i]) + gap * i for i in range(len(q_lens) + 1)], [sum(k_lens[:i]) + gap * i for i in range(len(k_lens) + 1)]
    q, do = ref.bf16(gen, qo[-1], hq * dim, std, pad, dev), ref.bf16(gen, qo[-1], hq * dim, 1e-3, 0, dev)
    k, v = ref.bf16(gen, ko[-1], hk * dim, std, pad, dev), ref.bf16(gen, ko[-1], hk * dim, 1.0, 2 * pad, dev)
    qs, ks = ref.spans(qo, q_lens), ref.spans(ko, k_lens)
    # the forward's results as a program keeps them: rounded from the exact ones
    o, _, lse, _ = ref.attention(q, k, v, dim, qs, ks, scale, causal)
    o, lse = o.to(torch.bfloat16).to(dev), lse.float().to(dev)
    if gap:
        for t, ss, off in ((q, qs, qo), (do, qs, qo), (k, ks, ko), (v, ks, ko)):
            for s, end in zip(ss, off[1:]):
                t[s.stop:end] = float("nan")
    kw = {"q_lengths": ref.i32(q_lens, dev), "k_lengths": ref.i32(k_lens, dev)} if gap else {}
    kw |= {"causal": causal, "scale": scale}
    return (do, q, k, v, o, lse, dim, ref.i32(qo, dev), ref.i32(ko, dev), max(q_lens) + loose,
            max(k_lens) + loose), kw, qs, ks


def nan_like(t, pad=0):
    return torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)[:, :t.shape[1]]


def run(dev, *a, **kw):
    args, call, qs, ks = case(dev, *a, **kw)
    do, q, k, v, o, lse, dim = args[:7]
    outs = {"dq": nan_like(q, 16), "dk": nan_like(k), "dv": nan_like(v, 32)}
    got = pf.puro_fp8_attention_bwd(*args, **call, **outs)
    torch.cuda.synchronize()
    want = ref.attention_bwd(do, q, k, v, o, lse, dim, qs, ks, call["scale"], call["causal"])
    for name, g, (w, tol) in zip(("dq", "dk", "dv"), got, want):
        assert g.data_ptr() == outs[name].data_ptr()
        ref.close_bf16(g, w, tol, (name, a, kw))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 129, 255, 257, 300, 513])
def test_one_sequence(dev, n, causal, dim):
    run(dev, 2, 1, dim, [n], [n], causal, seed=n)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 3), (16, 8), (12, 2), (33, 1)])
def test_heads(dev, hq, hk, causal, dim):
    run(dev, hq, hk, dim, [70, 5], [70, 131], causal, seed=hq)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q,k", [(1, 700), (3, 65), (40, 300), (300, 20), (40, 0), (64, 63), (257, 255), (700, 129), (130, 1000)])
def test_other_key_counts(dev, q, k, causal, dim):
    run(dev, 4, 2, dim, [q], [k], causal, seed=q + k)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("gap", [0, 3])
def test_packed(dev, causal, dim, gap):
    """Empty sequences of either kind: their keys' gradients are zero, rows of no sequence stay as they were."""
    lens = [5, 0, 130, 1, 64, 257, 0, 33]
    run(dev, 4, 2, dim, lens, lens, causal, seed=1, pad=16, gap=gap)
    run(dev, 4, 2, dim, lens, [9, 4, 130, 0, 90, 300, 0, 32], causal, seed=2, pad=32, gap=gap)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("scale,std", [(1.0, 1.0), (1e-4, 1.0), (0.125, 6.0)])
def test_scales(dev, dim, scale, std):
    run(dev, 2, 1, dim, [150], [150], True, seed=7, scale=scale, std=std)


@pytest.mark.parametrize("dim,causal", [(64, True), (128, False)])
def test_against_differences(dev, dim, causal):
    """d/dt of sum do o(q + t x, k + t y, v + t z) by central differences of the 64-bit forward."""
    q_lens, k_lens, hq, hk = [37, 20], [37, 64], 4, 2
    args, kw, qs, ks = case(dev, hq, hk, dim, q_lens, k_lens, causal, seed=21)
    do, q, k, v = args[:4]
    got = [ref.f64(t) for t in pf.puro_fp8_attention_bwd(*args, **kw)]
    bounds = ref.attention_bwd(do, q, k, v, *args[4:7], qs, ks, kw["scale"], causal)
    gen = torch.Generator().manual_seed(22)
    base = [ref.f64(t) for t in (q, k, v)]
    for which in range(3):
        x = torch.randn(base[which].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        loss = []
        for sign in (1, -1):
            moved = list(base)
            moved[which] = base[which] + sign * h * x
            loss.append(float((ref.f64(do) * ref.attention(*moved, dim, qs, ks, kw["scale"], causal)[0]).sum()))
        slope = (loss[0] - loss[1]) / (2 * h)
        w, tol = bounds[which]
        # the bound of every element and its BF16 rounding; o enters the gradient rounded to BF16, which moves
        # D by at most half a step of |do . o|; the difference's own error is of order h^2
        allowed = float(((tol + ref.B * w.abs()) * x.abs()).sum()) + float((ref.B * w.abs() * x.abs()).sum()) + 1e-9
        assert abs(float((got[which] * x).sum()) - slope) <= allowed, (which, slope)


def test_joint_gradient_and_equal_bits(dev):
    """dq, dk and dv as columns of one tensor; a workspace of any contents; the same bits every time."""
    args, kw, _, _ = case(dev, 4, 2, 64, [300, 77], [300, 77], True, seed=31)
    a = pf.puro_fp8_attention_bwd(*args, **kw)
    joint = torch.full((377, 8 * 64), float("nan"), dtype=torch.bfloat16, device=dev)
    for _ in range(3):
        ws = torch.full((1 << 22,), 0xFF, dtype=torch.uint8, device=dev)
        b = pf.puro_fp8_attention_bwd(*args, **kw, dq=joint[:, :256], dk=joint[:, 256:384], dv=joint[:, 384:], workspace=ws)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_nothing_to_do(dev):
    q, k = torch.empty((0, 128), dtype=torch.bfloat16, device=dev), torch.empty((0, 64), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((2, 0), device=dev)
    dq, dk, dv = pf.puro_fp8_attention_bwd(q, q, k, k, q, lse, 64, ref.i32([0], dev), ref.i32([0], dev), 0, 0)
    assert dq.shape == (0, 128) and dk.shape == (0, 64) and dv.shape == (0, 64)
    gen = torch.Generator().manual_seed(1)
    kk = ref.bf16(gen, 70, 64, 1.0, 0, dev)
    dq, dk, dv = pf.puro_fp8_attention_bwd(q, q, kk, kk, q, lse, 64, ref.i32([0, 0], dev), ref.i32([0, 70], dev), 0, 70)
    torch.cuda.synchronize()
    assert not dk.any() and not dv.any()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", [20, 300])
def test_nan_is_not_hidden(dev, n, dim):
    """A row whose lse is NaN has a NaN dq, and so have dk and dv of the keys that it sees."""
    args, kw, _, _ = case(dev, 2, 2, dim, [n], [n], True, seed=n)
    lse, row = args[5], n // 2
    lse[0, row] = float("nan")
    dq, dk, dv = pf.puro_fp8_attention_bwd(*args, **kw)
    torch.cuda.synchronize()
    assert bool(torch.isnan(dq[row, :dim]).all())
    assert bool(torch.isnan(dk[:row + 1, :dim]).all()) and bool(torch.isnan(dv[:row + 1, :dim]).all())
    others = torch.ones(n, dtype=torch.bool)
    others[row] = False
    assert bool(torch.isfinite(dq[others.to(dev)]).all()) and bool(torch.isfinite(dk[:, dim:]).all())


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q,k", [(100, 70), (70, 100), (40, 32), (200, 20), (33, 65), (5, 31), (300, 33)])
def test_rows_that_see_few_keys(dev, q, k, causal, dim):
    """Both sides of the 32 keys where D's form changes, inside a wave's 32 rows and between them."""
    run(dev, 6, 2, dim, [q, 3, q], [k, k, 4], causal, seed=q + k)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("times", [2, 3, 6])
def test_many_packed_rows(dev, times, causal, dim):
    """About 240, 360 and 720 workgroups of 128 rows or keys: every form of both kernels' workgroups."""
    lens = [300, 299, 257, 300, 129] * times
    run(dev, 8, 8, dim, lens, lens, causal, seed=times, gap=2)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q,k", [(1700, 1700), (130, 2049), (2100, 300)])
def test_long_rows(dev, q, k, dim):
    run(dev, 2, 1, dim, [q], [k], True, seed=q)
