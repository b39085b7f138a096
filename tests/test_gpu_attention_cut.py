"""Sequences that are longer than max_q, max_k or their tensor: the rows past the limit are left out, and those that
are kept see what they would see in the whole sequence (causal: query i the keys up to i + m - n, with the whole
sequence's n and m)."""
import pytest
import torch

import attn_ref as ref
import blockwise_fp8_gemm_amd as pf

pytestmark = pytest.mark.gpu

HQ, HK = 4, 2


def aligned(monkeypatch, shift):
    """The references' causal rows see j <= i + shift, whatever rows there are."""
    monkeypatch.setattr(ref, "hidden", lambda n, m, causal: torch.ones((n, m), dtype=torch.bool).triu(shift + 1)
                        if causal else torch.zeros((n, m), dtype=torch.bool))


def check(dev, monkeypatch, dim, causal, n, m, kept_q, kept_k, tokens_q, tokens_k, max_q, max_k, lengths, start_q=0, start_k=0):
    """One sequence of n queries and m keys, of which the first kept ones count, in tensors of tokens_q and tokens_k rows."""
    gen = torch.Generator().manual_seed(n + 7 * m + max_q)
    q, do = ref.bf16(gen, tokens_q, HQ * dim, 1.0, 0, dev), ref.bf16(gen, tokens_q, HQ * dim, 1e-3, 0, dev)
    k, v = ref.bf16(gen, tokens_k, HK * dim, 1.0, 0, dev), ref.bf16(gen, tokens_k, HK * dim, 1.0, 0, dev)
    qs, ks = [slice(start_q, start_q + kept_q)], [slice(start_k, start_k + kept_k)]
    for t, s in ((q, qs[0]), (do, qs[0]), (k, ks[0]), (v, ks[0])):      # rows that are left out reach nothing
        t[:s.start], t[s.stop:] = float("nan"), float("nan")
    if lengths:
        plan, kw = (dim, ref.i32([start_q], dev), ref.i32([start_k], dev), max_q, max_k), {"q_lengths": ref.i32([n], dev),
                                                                                         "k_lengths": ref.i32([m], dev)}
    else:
        plan, kw = (dim, ref.i32([start_q, start_q + n], dev), ref.i32([start_k, start_k + m], dev), max_q, max_k), {}
    nan = lambda t: torch.full_like(t, float("nan"))  # noqa: E731
    lse = torch.full((HQ, tokens_q), float("nan"), device=dev)
    o, _ = pf.puro_fp8_attention(q, k, v, *plan, causal=causal, o=nan(q), lse=lse, **kw)
    torch.cuda.synchronize()
    aligned(monkeypatch, m - n)
    want, tol, wl, lt = ref.attention(q, k, v, dim, qs, ks, dim ** -0.5, causal)
    ref.close_bf16(o, want, tol, "o")
    got = ref.f64(lse)
    assert torch.equal(torch.isnan(got), torch.isnan(wl))
    seen = torch.isfinite(wl)
    assert torch.equal(got[torch.isinf(wl)], wl[torch.isinf(wl)]) and bool(((got - wl).abs()[seen] <= lt[seen]).all())
    res = pf.puro_fp8_attention_bwd(do, q, k, v, o, lse, *plan, causal=causal, dq=nan(q), dk=nan(k), dv=nan(v), **kw)
    torch.cuda.synchronize()
    for g, (w, t), what in zip(res, ref.attention_bwd(do, q, k, v, o, lse, dim, qs, ks, dim ** -0.5, causal), ("dq", "dk", "dv")):
        ref.close_bf16(g, w, t, what)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lengths", [True, False])
@pytest.mark.parametrize("n,m,max_q,max_k", [(100, 100, 40, 100), (100, 100, 100, 50), (100, 100, 40, 50), (300, 300, 299, 270),
                                             (12, 200, 5, 200), (12, 200, 12, 150), (12, 200, 5, 20), (1, 3000, 1, 2500),
                                             (700, 4000, 600, 3900), (200, 90, 150, 80), (200, 20, 190, 20), (200, 20, 100, 20),
                                             (100, 400, 100, 30), (1000, 1000, 300, 1000)])
def test_past_a_maximum(dev, monkeypatch, n, m, max_q, max_k, lengths, causal, dim):
    check(dev, monkeypatch, dim, causal, n, m, min(n, max_q), min(m, max_k), n + 5, m + 9, max_q, max_k, lengths, 3, 6)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lengths", [True, False])
@pytest.mark.parametrize("n,m,tokens_q,tokens_k", [(100, 100, 60, 110), (100, 100, 110, 60), (100, 100, 60, 60), (2 ** 29, 70, 70, 70),
                                                   (70, 2 ** 29, 70, 70), (3, 900, 2, 700)])
def test_past_the_tensor(dev, monkeypatch, n, m, tokens_q, tokens_k, lengths, causal, dim):
    check(dev, monkeypatch, dim, causal, n, m, min(n, tokens_q), min(m, tokens_k), tokens_q, tokens_k, n if n < 2 ** 23 else 2 ** 23,
          m if m < 2 ** 23 else 2 ** 23, lengths)
