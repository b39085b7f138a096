"""Attention's running maximum where the first keys of a row lie a little below all the others: less than the 2^8 that
may be between a maximum and a score, but so many of them that every tile's sum is large."""
import pytest
import torch

import attn_ref as ref
import blockwise_fp8_gemm_amd as pf

pytestmark = pytest.mark.gpu

STEP = 4.84375      # a BF16 number, 6.99 in log2 units


def step_up(dev, hq, hk, dim, q_len, k_len, low):
    """Scores q . k of 0 for keys with low, of STEP for the others, in every row."""
    gen = torch.Generator().manual_seed(q_len)
    q = torch.zeros((q_len, hq * dim), dtype=torch.bfloat16, device=dev)
    q[:, ::dim] = 1.0
    k, v = ref.bf16(gen, k_len, hk * dim, 1.0, 0, dev), ref.bf16(gen, k_len, hk * dim, 1.0, 0, dev)
    for h in range(hk):
        k[:, h * dim] = torch.where(low, 0.0, STEP).to(torch.bfloat16).to(dev)
    return q, k, v


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hk,q_len,k_len", [(2, 1, 700, 700), (16, 8, 2, 300), (16, 8, 1100, 1100), (4, 4, 64, 9000)])
def test_first_keys_below_the_others(dev, hq, hk, q_len, k_len, causal, dim):
    q, k, v = step_up(dev, hq, hk, dim, q_len, k_len, torch.arange(k_len) < 128)
    o, lse = pf.puro_fp8_attention(q, k, v, dim, ref.i32([0, q_len], dev), ref.i32([0, k_len], dev), q_len, k_len,
                                   causal=causal, scale=1.0)
    torch.cuda.synchronize()
    want, tol, wl, lt = ref.attention(q, k, v, dim, [slice(0, q_len)], [slice(0, k_len)], 1.0, causal)
    ref.close_bf16(o, want, tol, "o")
    assert bool(((ref.f64(lse) - wl).abs() <= lt).all())


@pytest.mark.parametrize("hq,q_len,keys,waves", [(2, 64, 64, 1), (32, 1, 32, 2)])
def test_the_maximum_follows(dev, hq, q_len, keys, waves):
    """A share of the key axis leaves its maximum and sum in the workspace ([share][head][row] pairs, after the shares'
    outputs).  With heads of 128 the maximum is raised where a tile's sum shows that it lies too low; it then has to go all
    the way up, or the next tile's sum shows the same again, and every tile after it.  keys: of a tile; waves: of a share,
    with tiles of their own."""
    dim, k_len = 128, 9000
    plan = (dim, ref.i32([0, q_len], dev), ref.i32([0, k_len], dev), q_len, k_len)
    need = pf.puro_fp8_attention_workspace_size(hq, 1, dim, 1, q_len, k_len, q_len, k_len)
    shares, rest = divmod(need, hq * q_len * (dim + 2) * 4)
    assert shares > 1 and rest == 0
    # the first tile of every share and wave has the low keys
    tiles, parts = -(-k_len // keys), shares * waves
    low = torch.isin(torch.arange(k_len) // keys, torch.tensor([tiles * i // parts for i in range(parts)]))
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=dev)
    q, k, v = step_up(dev, hq, 1, dim, q_len, k_len, low)
    pf.puro_fp8_attention(q, k, v, *plan, causal=False, scale=1.0, workspace=ws)
    torch.cuda.synchronize()
    m, total = ws[shares * hq * q_len * dim * 4:].view(torch.float32).view(shares, hq * q_len, 2).double().cpu().unbind(2)
    top = torch.tensor(STEP, dtype=torch.float64) / torch.log(torch.tensor(2.0, dtype=torch.float64))
    # the product with the scale in log2 units: two roundings
    assert bool(((m - top).abs() <= top * 3 * ref.U).all()), m.unique()
    # each share has keys of either kind, and none counts for more than one
    assert bool((total < k_len).all()) and abs(float(total.sum(0)[0]) - float(torch.where(low, torch.exp2(-top), 1.0).sum())) < 1.0
