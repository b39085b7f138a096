"""puro_fp8_qk_norm_rope_bwd_quant_dual leaves what it does not turn as it is, to the sign of a zero: values' gradients in a
128-column tile that ends the key heads, and without weights the elements of a head behind the rotated ones."""
import pytest
import torch

import attn_ref as ref
import blockwise_fp8_gemm_amd as pf

pytestmark = pytest.mark.gpu


def with_zeros(gen, rows, cols, dev):
    """A third of the elements +0, a third -0."""
    x = ref.bf16(gen, rows, cols, 1e-3)
    kind = torch.randint(0, 3, (rows, cols), generator=gen)
    return torch.where(kind == 0, 0.0, torch.where(kind == 1, -0.0, x.float())).to(torch.bfloat16).to(dev)


def bits(t):
    return t.contiguous().view(torch.int16)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("tokens", [3, 256])
@pytest.mark.parametrize("dim,rotary,hq,hk", [(64, 64, 2, 1), (64, 32, 4, 3), (64, 16, 1, 2), (64, 0, 2, 1), (128, 64, 2, 1), (128, 48, 3, 2),
                                              (128, 128, 2, 1)])
def test_signs_of_zeros(dev, dim, rotary, hq, hk, tokens, norm, interleaved):
    gen = torch.Generator().manual_seed(dim + rotary + tokens)
    dq, dk, dv = (with_zeros(gen, tokens, h * dim, dev) for h in (hq, hk, hk))
    q, k = (ref.bf16(gen, tokens, h * dim, 1.0, 0, dev) for h in (hq, hk))
    w = torch.ones((dim,), device=dev) if norm else None
    pos = torch.arange(tokens, dtype=torch.int32, device=dev)
    freq = torch.linspace(0.1, 1.0, rotary // 2, device=dev) if rotary else None
    _, _, rstd = pf.puro_fp8_qk_norm_rope(q, k, dim, pos, freq, w, w, interleaved=interleaved)
    dx, _, _, qr, _, qt, _ = pf.puro_fp8_qk_norm_rope_bwd_quant_dual(dq, dk, dv, q, k, dim, pos, freq, rstd, w, w,
                                                                     interleaved=interleaved, store_dx=True)
    torch.cuda.synchronize()
    same = torch.zeros((hq + 2 * hk, dim), dtype=torch.bool)
    same[hq + hk:] = True
    if not norm:
        same[:, rotary:] = True
    same = same.flatten().to(dev)
    want = torch.cat((dq, dk, dv), 1)
    assert torch.equal(bits(dx)[:, same], bits(want)[:, same])
    sign = bits(want) < 0
    for codes in (qr, qt.t()):
        assert torch.equal((codes >= 128)[:, same], sign[:, same])
