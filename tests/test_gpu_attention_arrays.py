"""Offsets and lengths that no program should pass: whatever they hold, nothing outside the tensors is read or written.
A sequence that starts before the first row or behind the last one, or whose length is negative, has no rows; of one that
ends behind the last row those in the tensor count.  Guard rows of NaN lie before and behind every tensor."""
import pytest
import torch

import attn_ref as ref
import blockwise_fp8_gemm_amd as pf

pytestmark = pytest.mark.gpu

ROWS, GUARD, HQ, HK = 100, 40, 2, 1
LOW, HIGH = -2 ** 31, 2 ** 31 - 1

# (q_offsets, k_offsets) of one or two sequences, and lengths where they are given
WILD = [([-50, 2 ** 30], [0, 100], None, None), ([HIGH, LOW], [0, 100], None, None), ([LOW, HIGH], [0, 100], None, None),
        ([0, 100], [LOW, HIGH], None, None), ([0, 100], [-1, 99], None, None), ([0, 100], [99, HIGH], None, None),
        ([100, 100], [5, 3], None, None), ([101, HIGH], [0, 100], None, None), ([90, 70], [0, 50], None, None),
        ([-1, 40, 60], [0, 40, 60], None, None), ([0, 40, 60], [0, -40, 60], None, None), ([60, 100, HIGH], [0, 60, 200], None, None),
        ([-20, 50], [0, 50], [50, 50], [50, 50]), ([0, 50], [0, -50], [50, 50], [50, 100]), ([0, 50], [0, 50], [-1, LOW], [50, 50]),
        ([0, 50], [0, 50], [50, 50], [LOW, 40]), ([0, 99], [0, HIGH], [50, HIGH], [50, HIGH]), ([LOW, LOW], [LOW, LOW], [HIGH, HIGH], [HIGH, HIGH])]


def kept(offsets, lengths, most):
    """(slices of the rows that count, whole lengths)."""
    n = len(lengths) if lengths is not None else len(offsets) - 1
    spans, whole = [], []
    for i in range(n):
        a, m = offsets[i], lengths[i] if lengths is not None else offsets[i + 1] - offsets[i]
        m = 0 if a < 0 or a > ROWS else max(m, 0)
        a = min(max(a, 0), ROWS)
        spans.append(slice(a, a + min(m, ROWS - a, most)))
        whole.append(m)
    return spans, whole


def guarded(dev, t, dtype=torch.bfloat16):
    """t [ROWS][..] (None: NaN) between guard rows: (all of it, its middle)."""
    cols = t.shape[1]
    buf = torch.full((ROWS + 2 * GUARD, cols), float("nan"), dtype=dtype, device=dev)
    return buf, buf[GUARD:GUARD + ROWS]


def close(got, want, tol, what):
    """Every element within its bound, and the whole within half a step, as everywhere.  Where each row sees a single key
    the whole has no such measure: P = 1 and D = dP make dS, dq and dk zero, and the 64-bit formula with an lse rounded to
    FP32 leaves numbers of the order of that rounding, below their own bounds; then the elements' bounds stand alone."""
    fine = ~torch.isnan(want)
    if bool((want.abs() <= tol)[fine].all()):
        for i in range(want.shape[0]):
            ref.close_bf16(got[i:i + 1], want[i:i + 1], tol[i:i + 1], (what, i))
    else:
        ref.close_bf16(got, want, tol, what)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("most", [100, 16, 1])
@pytest.mark.parametrize("qo,ko,ql,kl", WILD)
def test_wild_arrays(dev, monkeypatch, qo, ko, ql, kl, most, causal, dim):
    gen = torch.Generator().manual_seed(5)
    ins, outs, whole_bufs = [], [], []
    for heads, std in ((HQ, 1.0), (HK, 1.0), (HK, 1.0), (HQ, 1e-3)):      # q, k, v, do; then o, dq, dk, dv
        x = ref.bf16(gen, ROWS, heads * dim, std, 0, dev)
        buf, mid = guarded(dev, x)
        mid.copy_(x)
        ins.append(mid)
    for heads in (HQ, HQ, HK, HK):
        buf, mid = guarded(dev, torch.empty((ROWS, heads * dim)))
        outs.append(mid)
        whole_bufs.append(buf)
    q, k, v, do = ins
    o, dq, dk, dv = outs
    lse_all = torch.full((HQ * ROWS + 2 * GUARD,), float("nan"), device=dev)
    lse = lse_all[GUARD:GUARD + HQ * ROWS].view(HQ, ROWS)
    kw = {"causal": causal, **({"q_lengths": ref.i32(ql, dev), "k_lengths": ref.i32(kl, dev)} if ql else {})}
    plan = (dim, ref.i32(qo, dev), ref.i32(ko, dev), most, ROWS)
    pf.puro_fp8_attention(q, k, v, *plan, o=o, lse=lse, **kw)
    torch.cuda.synchronize()
    (qs, qn), (ks, kn) = kept(qo, ql, most), kept(ko, kl, ROWS)
    want = torch.full((ROWS, HQ * dim), float("nan"), dtype=torch.float64)
    wl = torch.full((HQ, ROWS), float("nan"), dtype=torch.float64)
    tol, lt, bounds = torch.zeros_like(want), torch.zeros_like(wl), []
    for s, (a, b) in enumerate(zip(qs, ks)):      # one sequence at a time: each has a mask of its own
        shift = kn[s] - qn[s]
        monkeypatch.setattr(ref, "hidden", lambda n, m, c, shift=shift: (torch.arange(m) > torch.arange(n)[:, None] + shift) & c)
        x, t, y, u = ref.attention(q, k, v, dim, [a], [b], dim ** -0.5, causal)
        want[a], tol[a], wl[:, a], lt[:, a] = x[a], t[a], y[:, a], u[:, a]
    ref.close_bf16(o, want, tol, "o")
    got = ref.f64(lse)
    assert torch.equal(torch.isnan(got), torch.isnan(wl)) and torch.equal(torch.isinf(got), torch.isinf(wl))
    fine = torch.isfinite(wl)
    assert bool(((got - wl).abs()[fine] <= lt[fine]).all())

    pf.puro_fp8_attention_bwd(do, q, k, v, o, lse, *plan, dq=dq, dk=dk, dv=dv, **kw)
    torch.cuda.synchronize()
    want = [torch.full((ROWS, h * dim), float("nan"), dtype=torch.float64) for h in (HQ, HK, HK)]
    tols = [torch.zeros_like(w) for w in want]
    for s, (a, b) in enumerate(zip(qs, ks)):
        shift = kn[s] - qn[s]
        monkeypatch.setattr(ref, "hidden", lambda n, m, c, shift=shift: (torch.arange(m) > torch.arange(n)[:, None] + shift) & c)
        res = ref.attention_bwd(do, q, k, v, torch.nan_to_num(o), lse, dim, [a], [b], dim ** -0.5, causal)
        for i, rows in enumerate((a, b, b)):
            want[i][rows], tols[i][rows] = res[i][0][rows], res[i][1][rows]
    for g, w, t, what in zip((dq, dk, dv), want, tols, ("dq", "dk", "dv")):
        close(g, w, t, what)
    for buf in whole_bufs:
        assert bool(torch.isnan(buf[:GUARD]).all()) and bool(torch.isnan(buf[GUARD + ROWS:]).all())
    assert bool(torch.isnan(lse_all[:GUARD]).all()) and bool(torch.isnan(lse_all[GUARD + HQ * ROWS:]).all())
